"""GPU parity of block-sparse attention and the passes in front of it against the
float64 oracle, through the binding and the C ABI.

Tolerances are element-wise bounds from the arithmetic: a rounding to a 16-bit
type is off by at most half a step (bf16 2^-8, fp16 2^-11 of the value, fp16
below 2^-14 by 2^-25 absolutely), one to fp32 by 2^-24."""

import ctypes
import math
import os
import subprocess
import sys
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import oracle as orc
import partitioned_attention_state_b200 as dt
from oracle import sparse as sp
from partitioned_attention_state_b200.session import Session

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF: 0.0, FP: 2.0 ** -25, F32: 0.0}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def np64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def within(got, ref, bound, what):
    got, bad = np64(got), None
    assert got.shape == ref.shape, what
    fin = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), fin) and np.array_equal(got[~fin], ref[~fin]), f"{what}: non-finite pattern"
    over = np.abs(got[fin] - ref[fin]) - np.broadcast_to(bound, ref.shape)[fin]
    if over.size and over.max() > 0:
        bad = over.max()
    assert bad is None, f"{what}: {(over > 0).sum()} of {over.size} beyond the bound, worst by {bad:.3e}"


# ------------------------------------------------------------------ rope table
@pytest.mark.parametrize("S,axes,far", [(1, (2,), 0), (7, (6,), 5), (1024, (36, 36), 0), (33, (44, 42, 42), 1 << 20),
                                        (5, (128,), (1 << 31) - 9), (100, (2, 4, 6, 8), -50), (3, (256,), 131072)])
def test_rope_table(S, axes, far):
    g = np.random.Generator(np.random.PCG64(S))
    pos = g.integers(0, 4, (len(axes), S)) + np.arange(S) + far
    pos = np.minimum(pos, (1 << 31) - 1).astype(np.int32)
    n = sum(axes) // 2
    buf = torch.full((S * n * 2 + 64,), 7.0, device="cuda")
    table = buf[:S * n * 2].view(S, n, 2)
    dt.dt_rope_table(dt.rope_params(S, axes), torch.from_numpy(pos).cuda(), table)
    ref, turns = sp.rope_table(pos, axes)
    # sine and cosine of the fraction (1 ulp of at most 1), the correction and its rounding, and the
    # 64-bit angle's own error: three roundings of |turns|, times 2 pi, on each side
    within(table, ref, 2.0 ** -22 + 2 * np.pi * 2 * 4 * 2.0 ** -53 * np.abs(turns)[..., None], "table")
    assert bool((buf[S * n * 2:] == 7.0).all())


# ------------------------------------------------------------------ norm + rotation
def norm_case(S, H, Hkv, D, rot, halves, ity, oty, norm=True, weights=True, blocks=(128, 64), seed=0):
    g = gen(seed)
    x = randn(g, S, H + 2 * Hkv, D, dtype=ity) * 3
    wq, wk = (1 + 0.2 * randn(g, D), 1 + 0.2 * randn(g, D)) if weights else (None, None)
    ang = torch.rand(S, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 100
    table = torch.stack([ang.cos(), ang.sin()], -1).float() if rot else None
    xt = x.transpose(0, 1)
    q, k, v = xt[:H], xt[H:H + Hkv], xt[H + Hkv:]
    # one row more than the sequence behind every output: it has to stay
    outs = [torch.full((n, S + 1, D), 9.0, dtype=oty, device="cuda") for n in (H, Hkv, Hkv)]
    Q, K, V = (t[:, :S] for t in outs)
    nq, nk = -(-S // blocks[0]), -(-S // blocks[1])
    qm, km = torch.full((H, nq, D), 9.0, device="cuda"), torch.full((Hkv, nk, D), 9.0, device="cuda")
    p = dt.norm_rope_params(q, k, v, Q, K, V, rot=rot, pairing=int(halves), norm=norm, q_block=blocks[0], k_block=blocks[1])
    dt.dt_qk_norm_rope(p, q, k, v, wq, wk, table, Q, K, V, qm, km)
    for name, src, w, out, m, blk in (("Q", q, wq, Q, qm, blocks[0]), ("K", k, wk, K, km, blocks[1])):
        y, mag = sp.norm_rope(np64(src), None if w is None else np64(w), None if table is None else np64(table), halves, norm)
        # fp32: the sum of squares (D/8 + 3 roundings at most 19 in a row), division, reciprocal root (2 ulp),
        # two scalings and the rotation's two products and sum stay below 2^-19 of the absolute terms
        arith = 2.0 ** -19 * mag if (norm or rot) else 0 * mag
        within(out, y, arith + HALF[oty] * (np.abs(y) + arith) + TINY[oty], name)
        # the mean adds at most 128 such values one after another
        mm = sp.block_means(mag, blk)
        within(m, sp.block_means(y, blk), (2.0 ** -19 + 128 * 2.0 ** -24) * mm, name + " mean")
    ref = np64(v)
    within(V, ref, HALF[oty] * np.abs(ref) + TINY[oty] if oty != ity else 0 * ref, "V")
    for t in outs:
        assert bool((t[:, S] == 9.0).all())


@pytest.mark.parametrize("S", [1, 2, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (72, 72), (128, 128), (128, 64), (72, 24)])
def test_norm_rope_sizes(S, halves, D, rot):
    norm_case(S, 3, 2, D, rot, halves, BF, BF, seed=S)


@pytest.mark.parametrize("ity,oty", [(BF, BF), (FP, FP), (F32, F32), (FP, BF), (F32, BF)])
@pytest.mark.parametrize("blocks", [(128, 64), (64, 128)])
@pytest.mark.parametrize("D,rot,halves", [(64, 64, True), (72, 72, False), (8, 8, True), (40, 0, False), (128, 120, True)])
def test_norm_rope_types_and_blocks(ity, oty, blocks, D, rot, halves):
    norm_case(200, 2, 1, D, rot, halves, ity, oty, blocks=blocks, seed=3)


@pytest.mark.parametrize("norm,weights,rot", [(False, False, 0), (False, False, 64), (True, False, 0), (True, True, 0)])
def test_norm_rope_parts_of_the_work(norm, weights, rot):
    norm_case(150, 2, 2, 64, rot, False, BF, BF, norm=norm, weights=weights, seed=5)


def test_norm_rope_many_heads_share_a_cta():
    norm_case(2100, 40, 40, 128, 128, False, BF, BF, seed=6)


def test_norm_rope_one_token_into_a_longer_cache_and_in_place():
    g = gen(7)
    H, D, S = 5, 128, 1
    x = randn(g, S, 3 * H, D, dtype=BF)
    q, k, v = (x.transpose(0, 1)[i * H:(i + 1) * H] for i in range(3))
    cache = torch.zeros(2, H, 300, D, dtype=BF, device="cuda")
    ang = torch.rand(S, D // 2, generator=g, device="cuda")
    table = torch.stack([ang.cos(), ang.sin()], -1)
    Q = torch.empty(H, S, D, dtype=BF, device="cuda")
    p = dt.norm_rope_params(q, k, v, Q, cache[0][:, 211:212], cache[1][:, 211:212], rot=D, pairing=dt.DT_ROPE_HALVES)
    dt.dt_qk_norm_rope(p, q, k, v, None, None, table, Q, cache[0][:, 211:212], cache[1][:, 211:212])
    want = cache.clone()
    assert bool((cache[:, :, :211] == 0).all()) and bool((cache[:, :, 212:] == 0).all())
    assert torch.equal(cache[1][:, 211], v[:, 0]) and bool((cache[0][:, 211] != 0).any())
    # in place: the same result over the input's own memory
    y = x.clone()
    yq, yk = (y.transpose(0, 1)[i * H:(i + 1) * H] for i in range(2))
    p = dt.norm_rope_params(yq, yk, None, yq, yk, None, rot=D, pairing=dt.DT_ROPE_HALVES)
    dt.dt_qk_norm_rope(p, yq, yk, None, None, None, table, yq, yk, None)
    assert torch.equal(yq, Q) and torch.equal(yk, want[0][:, 211:212])
    assert torch.equal(y[:, 2 * H:], x[:, 2 * H:])


@pytest.mark.parametrize("ty", [BF, FP, F32])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("S,H,Hkv,D", [(1, 3, 1, 64), (333, 3, 3, 72), (2500, 24, 8, 128)])
def test_norm_rope_in_place_equals_out_of_place(ty, halves, S, H, Hkv, D):
    """Packed token-major tensors normalised over themselves, at sizes with one and with many warps per head."""
    g = gen(S)
    x = randn(g, S, H + 2 * Hkv, D, dtype=ty)
    t = x.transpose(0, 1)
    ang = torch.rand(S, D // 2, generator=g, device="cuda")
    table = torch.stack([ang.cos(), ang.sin()], -1)
    w = 1 + 0.1 * randn(g, D)
    Q, K = torch.empty(H, S, D, dtype=ty, device="cuda"), torch.empty(Hkv, S, D, dtype=ty, device="cuda")
    p = dt.norm_rope_params(t[:H], t[H:H + Hkv], None, Q, K, None, rot=D, pairing=int(halves))
    dt.dt_qk_norm_rope(p, t[:H], t[H:H + Hkv], None, w, w, table, Q, K, None)
    y = x.clone()
    u = y.transpose(0, 1)
    qm, km = torch.empty(H, -(-S // 128), D, device="cuda"), torch.empty(Hkv, -(-S // 64), D, device="cuda")
    p = dt.norm_rope_params(u[:H], u[H:H + Hkv], None, u[:H], u[H:H + Hkv], None, rot=D, pairing=int(halves))
    dt.dt_qk_norm_rope(p, u[:H], u[H:H + Hkv], None, w, w, table, u[:H], u[H:H + Hkv], None, qm, km)
    assert torch.equal(u[:H], Q) and torch.equal(u[H:H + Hkv], K) and torch.equal(y[:, H + Hkv:], x[:, H + Hkv:])


def test_norm_rope_offsets_past_32_bits():
    """An input and an output of more than 2^31 elements each: rows at both ends against the oracle."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = gen(25)
    S, H, D = 700_001, 26, 128
    x = torch.empty(S, H, D, dtype=BF, device="cuda")
    for a in range(0, S, 100_000):
        x[a:a + 100_000] = randn(g, min(100_000, S - a), H, D, dtype=BF)
    t = x.transpose(0, 1)
    ang = torch.rand(S, 8, generator=g, device="cuda") * 6
    table = torch.stack([ang.cos(), ang.sin()], -1)
    Q, qm = torch.empty(H, S, D, dtype=BF, device="cuda"), torch.empty(H, -(-S // 128), D, device="cuda")
    assert x.numel() > 1 << 31 and Q.numel() > 1 << 31
    p = dt.norm_rope_params(t, Q=Q, rot=16)
    dt.dt_qk_norm_rope(p, t, None, None, None, None, table, Q, None, None, qm)
    for h, a in ((0, 0), (H - 1, 0), (0, S - 65), (H - 1, S - 65), (13, 350_000 // 128 * 128)):
        y, mag = sp.norm_rope(np64(t[h:h + 1, a:a + 65]), None, np64(table[a:a + 65]))
        within(Q[h:h + 1, a:a + 65], y, 2.0 ** -19 * mag + HALF[BF] * (np.abs(y) + 2.0 ** -19 * mag), f"rows {a} of head {h}")
    last = S // 128 * 128
    y, mag = sp.norm_rope(np64(t[H - 1:, last:]), None, np64(table[last:]))
    within(qm[H - 1:, -1:], sp.block_means(y, 128), (2.0 ** -19 + 128 * 2.0 ** -24) * sp.block_means(mag, 128), "last mean")


def test_norm_and_select_at_once_on_two_streams():
    g = gen(26)
    q, k = randn(g, 8, 1000, 128, dtype=BF), randn(g, 8, 1000, 128, dtype=BF)
    ang = torch.rand(1000, 64, generator=g, device="cuda")
    table = torch.stack([ang.cos(), ang.sin()], -1)
    out = []
    torch.cuda.synchronize()
    for s in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        Q, K = torch.empty_like(q), torch.empty_like(k)
        qm, km = torch.empty(8, 8, 128, device="cuda"), torch.empty(8, 16, 128, device="cuda")
        idx, count = torch.empty(8, 8, 5, dtype=torch.int32, device="cuda"), torch.empty(8, 8, dtype=torch.int32, device="cuda")
        out.append((Q, K, qm, km, idx, count, s))
    torch.cuda.synchronize()
    p = dt.norm_rope_params(q, k, None, out[0][0], out[0][1], None, rot=128)
    for Q, K, qm, km, idx, count, s in out:
        dt.dt_qk_norm_rope(p, q, k, None, None, None, table, Q, K, None, qm, km, s)
        dt.dt_block_select(dt.select_params(8, 8, 8, 16, 128, 5, 1, 0, 2.0), qm, km, idx, count, s)
    torch.cuda.synchronize()
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0][:6], other[:6]))


def test_norm_rope_odd_head_counts_mix_parts_in_a_warp():
    """Heads of all parts share warps when the counts are odd; infinities in one head stay there."""
    norm_case(130, 5, 3, 64, 64, False, BF, BF, seed=21)
    norm_case(130, 1, 1, 128, 64, True, FP, FP, seed=22)
    g = gen(23)
    x = randn(g, 70, 5, 64, dtype=BF)
    x[:, 1] = math.inf
    t = x.transpose(0, 1)
    q, k, v = t[:1], t[1:3], t[3:5]
    Q, K, V = (torch.empty(n, 70, 64, dtype=BF, device="cuda") for n in (1, 2, 2))
    p = dt.norm_rope_params(q, k, v, Q, K, V)
    dt.dt_qk_norm_rope(p, q, k, v, None, None, None, Q, K, V)
    assert bool(torch.isfinite(Q).all()) and bool(torch.isfinite(K[1]).all()) and torch.equal(V, v)


def test_norm_rope_means_alone_and_single_parts():
    g = gen(8)
    q = randn(g, 3, 500, 72, dtype=BF)
    qm = torch.empty(3, 4, 72, device="cuda")
    p = dt.norm_rope_params(q, norm=False)
    dt.dt_qk_norm_rope(p, q, None, None, None, None, None, None, None, None, qm)
    within(qm, sp.block_means(np64(q), 128), 128 * 2.0 ** -24 * sp.block_means(np.abs(np64(q)), 128), "mean")
    V = torch.empty(3, 500, 72, dtype=BF, device="cuda")
    p = dt.norm_rope_params(v=q, V=V)
    dt.dt_qk_norm_rope(p, None, None, q, None, None, None, None, None, V)
    assert torch.equal(V, q)


def test_norm_rope_zero_row_and_non_finite_rows_stay_apart():
    """A row of zeros normalises to zeros; an infinite or NaN row touches no other row and no mean but its own."""
    g = gen(9)
    q = randn(g, 1, 300, 64, dtype=BF)
    q[0, 5] = 0
    q[0, 200, 3], q[0, 201, 0] = math.inf, math.nan
    Q, qm = torch.empty_like(q), torch.empty(1, 3, 64, device="cuda")
    p = dt.norm_rope_params(q, Q=Q)
    dt.dt_qk_norm_rope(p, q, None, None, None, None, None, Q, None, None, qm)
    assert bool((Q[0, 5] == 0).all())
    rows = torch.isfinite(Q[0]).all(-1)
    assert rows.sum() == 298 and not rows[200] and not rows[201]
    assert bool(torch.isfinite(qm[0, 0]).all()) and bool(torch.isfinite(qm[0, 2]).all())


# ------------------------------------------------------------------ selection
def run_select(qm, km, topk, first=0, last=0, margin=math.inf):
    H, nq, D = qm.shape
    buf = torch.full((H * nq * topk + 32,), -7, dtype=torch.int32, device="cuda")
    idx = buf[:H * nq * topk].view(H, nq, topk)
    count = torch.full((H, nq), -7, dtype=torch.int32, device="cuda")
    p = dt.select_params(H, km.shape[0], nq, km.shape[1], D, topk, first, last, margin)
    dt.dt_block_select(p, qm, km, idx, count)
    assert bool((buf[H * nq * topk:] == -7).all())
    return idx.cpu().numpy(), count.cpu().numpy()


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (2, 31), (3, 32), (5, 33), (9, 64), (8, 65), (17, 200), (40, 513),
                                   (1, 3000), (3, 1500)])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_select_matches_oracle(nq, nk, D):
    g = gen(nq * 1000 + nk)
    qm, km = randn(g, 4, nq, D), randn(g, 2, nk, D)
    for topk, first, last, margin in {(1, 0, 0, math.inf), (max(1, nk // 3), 0, 0, math.inf),
                                      (min(nk, 7), 2 if nk > 7 else 0, 3 if nk > 7 else 0, 1.5), (nk, 0, 0, 0.5),
                                      (nk + 5, 1, 1, math.inf), (min(nk, 40), 0, 1, 0.0)}:
        got = run_select(qm, km, topk, first, last, margin)
        ref = sp.block_select(np64(qm), np64(km), topk, first, last, margin)
        np.testing.assert_array_equal(got[0], ref[0])
        np.testing.assert_array_equal(got[1], ref[1])


def test_select_largest_row():
    g = gen(2)
    qm, km = randn(g, 1, 2, 128), randn(g, 1, 16384, 128)
    got = run_select(qm, km, 100, 1, 1)
    ref = sp.block_select(np64(qm), np64(km), 100, 1, 1)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])


@pytest.mark.parametrize("kind", ["outlier", "clusters", "steps", "ulps", "huge", "tiny"])
@pytest.mark.parametrize("nk", [40, 300, 1000])
def test_select_uneven_scores(kind, nk):
    """Scores that crowd into one bin of the row's range, in every way the selection tells them apart."""
    g = gen(nk)
    qm = torch.zeros(2, 5, 64, device="cuda")
    qm[..., 0] = 1.0
    km = torch.zeros(1, nk, 64, device="cuda")
    x = torch.randn(nk, generator=g, device="cuda")
    if kind == "outlier":                            # one score far above: the rest share a bin
        x[nk // 2] = 1e9
    elif kind == "clusters":
        x = x * 1e-4 + torch.where(torch.arange(nk, device="cuda") % 3 == 0, 7.0, -2.0)
    elif kind == "steps":                            # few values, many ties
        x = torch.round(x * 2)
    elif kind == "ulps":
        x = 1.0 + torch.randint(0, 40, (nk,), generator=g, device="cuda") * 2.0 ** -23
    elif kind == "huge":                             # the range itself overflows fp32
        x = x * 1e38
        qm[..., 0] = 1e30
    else:
        x = x * 1e-38
        qm[..., 0] = 1e-30
    km[0, :, 0] = x
    for topk, first, last, margin in ((1, 0, 0, math.inf), (nk // 3, 0, 0, math.inf), (nk // 3, 3, 2, 0.25),
                                      (nk - 1, 0, 1, math.inf), (33, 33, 0, math.inf), (20, 0, 0, 1e-6)):
        if first + last > topk:
            continue
        got, ref = run_select(qm, km, topk, first, last, margin), sp.block_select(np64(qm), np64(km), topk, first, last, margin)
        np.testing.assert_array_equal(got[0], ref[0])
        np.testing.assert_array_equal(got[1], ref[1])


def test_select_equal_scores_take_the_lowest_indices():
    qm = torch.ones(1, 3, 64, device="cuda")
    km = torch.zeros(1, 100, 64, device="cuda")
    km[0, 10:90] = 1.0                              # eighty equal best scores
    km[0, 50:] *= -0.0                              # the rest: zeros of both signs, equal too
    idx, count = run_select(qm, km, 60)
    np.testing.assert_array_equal(idx[0, 0], list(range(0, 60)))
    assert (count == 60).all()
    idx, _ = run_select(qm, km, 7)
    np.testing.assert_array_equal(idx[0, 2], list(range(10, 17)))


def test_select_non_finite_scores():
    g = gen(3)
    qm, km = randn(g, 1, 2, 64), randn(g, 1, 40, 64)
    km[0, 3], km[0, 7], km[0, 9] = math.nan, math.inf, -math.inf        # inf times mixed signs: NaN too
    qm[0, 0] = qm[0, 0].abs()                       # row 0: +inf at 7, -inf at 9
    for topk, margin in ((5, math.inf), (40, math.inf), (39, math.inf), (10, 1.0), (40, 1.0)):
        got, ref = run_select(qm, km, topk, 0, 0, margin), sp.block_select(np64(qm), np64(km), topk, 0, 0, margin)
        np.testing.assert_array_equal(got[0], ref[0])
        np.testing.assert_array_equal(got[1], ref[1])
    km[:] = math.nan                                # nothing but NaN: the lowest indices
    np.testing.assert_array_equal(run_select(qm, km, 4)[0][0, 1], [0, 1, 2, 3])


def test_select_no_key_blocks_gives_empty_lists():
    idx, count = run_select(torch.ones(2, 3, 64, device="cuda"), torch.ones(1, 0, 64, device="cuda"), 4)
    assert (idx == -1).all() and (count == 0).all()


def test_select_keeps_scores_that_differ_in_the_last_bits_of_64():
    """Scores 1 and 1 + 2^-46: equal in fp32, told apart here."""
    qm, km = torch.zeros(1, 1, 64, device="cuda"), torch.zeros(1, 50, 64, device="cuda")
    qm[0, 0, 0], qm[0, 0, 1] = 1.0, 2.0 ** -23
    km[0, :, 0] = 1.0
    km[0, 31, 1] = 2.0 ** -23
    idx, _ = run_select(qm, km, 1)
    assert idx[0, 0, 0] == 31


# ------------------------------------------------------------------ attention
def lists_for(g, H, Sq, Sk, block, cap, counts):
    nq, nk = -(-Sq // 128), -(-Sk // block)
    count = np.asarray(counts(H, nq) if callable(counts) else np.full((H, nq), counts), np.int32)
    idx = torch.rand(H, nq, nk, generator=g, device="cuda").argsort(-1)[..., :cap].to(torch.int32)
    assert idx.shape[-1] == cap and (count <= cap).all()
    return idx.contiguous(), torch.from_numpy(count).cuda()


def attend(q, k, v, idx, count, block, oty=None, o=None, stream=None):
    H, Sq, D = q.shape
    guard = torch.full((H, Sq + 1, D), 9.0, dtype=oty or q.dtype, device="cuda")
    O = guard[:, :Sq] if o is None else o
    lg = torch.full((H * Sq + 4,), 9.0, device="cuda")
    L = lg[:H * Sq].view(H, Sq)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    p = dt.sparse_params(q, k, v, O, block, idx.shape[-1])
    dt.dt_attn_block_sparse(p, q, k, v, idx, count, O, L, st, stream)
    torch.cuda.synchronize()
    assert bool((guard[:, Sq] == 9.0).all()) and bool((lg[H * Sq:] == 9.0).all()), "rows behind the last"
    return O, L, int(st[0])


def check_attention(q, k, v, idx, count, block, O, L):
    ref_o, ref_l, A, s = sp.block_sparse_attention(np64(q), np64(k), np64(v), idx.cpu().numpy(), count.cpu().numpy(), block)
    D, n = q.shape[-1], idx.shape[-1] * block
    ty = q.dtype
    # logits: D products summed in fp32 with rounding or truncation, and the scaling to exponents (2^-22 of
    # |logit| <= s); a weight's relative error is the logit's absolute one, plus ex2's 2^-22; the row sum adds n weights
    e = s * (D * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -22 + n / 32 * 2.0 ** -24
    vmax = np.abs(np64(v)).max() if v.numel() else 0.0
    # O: P rounded to 16 bits (half a step of each weight; below fp16's normal range 2^-25 each, of a sum >= 1),
    # numerator and denominator off by e each, the tensor cores' fp32 sums over n keys, the output's rounding
    o = (HALF[ty] + 2 * e + n * 2.0 ** -24)[..., None] * A + TINY[ty] * n * vmax
    within(O, ref_o, o + HALF[O.dtype] * (np.abs(ref_o) + o) + TINY[O.dtype], "O")
    fl = np.where(np.isfinite(ref_l), np.abs(ref_l), 0)
    within(L, ref_l, e + 2.0 ** -22 * (1 + fl + s), "L")


RAGGED = lambda cap: (lambda H, nq: (5 * np.arange(H)[:, None] + 3 * np.arange(nq) + cap // 2) % (cap + 1))  # noqa: E731


@pytest.mark.parametrize("ty", [BF, FP])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("H,Hkv,Sq,Sk,block,cap", [
    (1, 1, 1, 1, 64, 1), (2, 1, 1, 100, 64, 2), (1, 1, 5, 64, 128, 1), (2, 2, 128, 129, 64, 3), (2, 1, 129, 200, 128, 2),
    (4, 2, 300, 1000, 64, 7), (3, 3, 257, 777, 128, 5), (1, 1, 1, 5000, 64, 79), (2, 1, 17, 4100, 128, 33)])
def test_attention_sizes(ty, D, H, Hkv, Sq, Sk, block, cap):
    g = gen(Sq + Sk)
    q, k, v = randn(g, H, Sq, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty)
    for counts in (cap, RAGGED(cap)):
        idx, count = lists_for(g, H, Sq, Sk, block, cap, counts)
        O, L, st = attend(q, k, v, idx, count, block)
        assert st == 0
        check_attention(q, k, v, idx, count, block, O, L)


@pytest.mark.parametrize("ty", [BF, FP])
@pytest.mark.parametrize("H,Hkv,Sq,D,block", [(40, 40, 600, 128, 64), (160, 20, 128, 64, 128), (30, 30, 700, 72, 64)])
def test_attention_many_items_per_cta(ty, H, Hkv, Sq, D, block):
    """More items than SMs: the persistent loop, Q double-buffered across items, empty and odd lists among them."""
    g = gen(11)
    Sk, cap = 1500, 9
    q, k, v = randn(g, H, Sq, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty)
    idx, count = lists_for(g, H, Sq, Sk, block, cap, RAGGED(cap))
    O, L, st = attend(q, k, v, idx, count, block)
    assert st == 0
    check_attention(q, k, v, idx, count, block, O, L)


@pytest.mark.parametrize("H,Sq,cap", [(1, 1, 64), (1, 1, 33), (3, 1, 47), (5, 130, 30), (9, 128, 63), (20, 100, 64), (37, 1, 64),
                                      (74, 3, 8), (75, 3, 8)])
@pytest.mark.parametrize("block", [64, 128])
def test_attention_lists_split_over_a_cluster(H, Sq, cap, block):
    g = gen(13)
    D, Sk = 128, 64 * block
    q, k, v = randn(g, H, Sq, D, dtype=BF), randn(g, 1, Sk, D, dtype=BF), randn(g, 1, Sk, D, dtype=BF)
    for counts in (cap, RAGGED(cap), 1):
        idx, count = lists_for(g, H, Sq, Sk, block, cap, counts)
        O, L, st = attend(q, k, v, idx, count, block)
        assert st == 0
        check_attention(q, k, v, idx, count, block, O, L)


def test_attention_large_logits_and_late_maxima():
    """Logits up to about 60, rising along the list: the running maximum moves again and again."""
    g = gen(17)
    H, Sq, Sk, D = 2, 200, 2048, 64
    q, k, v = randn(g, H, Sq, D), randn(g, H, Sk, D), randn(g, H, Sk, D, dtype=BF)
    q[..., 0], k[..., 0] = 20.0, torch.arange(Sk, device="cuda") * (24.0 / Sk)
    q, k = q.to(BF), k.to(BF)
    idx = torch.arange(32, device="cuda", dtype=torch.int32).expand(H, 2, 32).contiguous()
    count = torch.full((H, 2), 32, dtype=torch.int32, device="cuda")
    for order in (idx, idx.flip(-1).contiguous()):
        O, L, _ = attend(q, k, v, order, count, 64)
        check_attention(q, k, v, order, count, 64, O, L)


def test_attention_token_major_views_and_longer_caches():
    """Q, O token-major, K and V a prefix of a longer cache whose other rows are NaN; bit-identical to dense buffers."""
    g = gen(19)
    H, Hkv, Sq, Sk, D = 6, 3, 333, 700, 128
    qt = randn(g, Sq, H, D, dtype=BF)
    cache = torch.full((2, Hkv, 1000, D), math.nan, dtype=BF, device="cuda")
    cache[:, :, :Sk] = randn(g, 2, Hkv, Sk, D, dtype=BF)
    q, k, v = qt.transpose(0, 1), cache[0][:, :Sk], cache[1][:, :Sk]
    idx, count = lists_for(g, H, Sq, Sk, 64, 6, RAGGED(6))
    ot = torch.zeros(Sq, H, D, dtype=BF, device="cuda")
    O, L, st = attend(q, k, v, idx, count, 64, o=ot.transpose(0, 1))
    O2, L2, _ = attend(q.contiguous(), k.contiguous(), v.contiguous(), idx, count, 64)
    assert st == 0 and torch.equal(O, O2) and torch.equal(L, L2)
    check_attention(q, k, v, idx, count, 64, O, L)


def test_attention_on_the_packed_projection_itself():
    """Q, K and V as views of one token-major tensor, O token-major too."""
    g = gen(20)
    H, S, D = 5, 700, 72
    x = randn(g, S, 3, H, D, dtype=BF)
    q, k, v = (x[:, i].transpose(0, 1) for i in range(3))
    idx, count = lists_for(g, H, S, S, 64, 7, RAGGED(7))
    O, L, st = attend(q, k, v, idx, count, 64, o=torch.zeros(S, H, D, dtype=BF, device="cuda").transpose(0, 1))
    O2, L2, _ = attend(q.contiguous(), k.contiguous(), v.contiguous(), idx, count, 64)
    assert st == 0 and torch.equal(O, O2) and torch.equal(L, L2)
    check_attention(q, k, v, idx, count, 64, O, L)


@pytest.mark.parametrize("H,Sq,cap", [(300, 1, 3), (3, 6400, 2), (16, 1280, 5)])
def test_attention_many_short_lists(H, Sq, cap):
    """Items of no, one or two tiles: the scheduler, not the tiles, sets the pace."""
    g = gen(24)
    q, k, v = randn(g, H, Sq, 64, dtype=BF), randn(g, 1, 500, 64, dtype=BF), randn(g, 1, 500, 64, dtype=BF)
    for counts in (RAGGED(cap), 0, 1):
        idx, count = lists_for(g, H, Sq, 500, 64, cap, counts)
        O, L, st = attend(q, k, v, idx, count, 64)
        assert st == 0
        check_attention(q, k, v, idx, count, 64, O, L)


def test_attention_first_call_inside_a_capture():
    """A process whose first call of the kernel is captured: its one-time set-up is legal there."""
    code = (
        "import torch, partitioned_attention_state_b200 as dt\n"
        "q = torch.randn(2, 300, 64, device='cuda').half(); k = torch.randn(2, 256, 64, device='cuda').half()\n"
        "idx = torch.arange(4, device='cuda', dtype=torch.int32).expand(2, 3, 4).contiguous()\n"
        "O, L = torch.zeros_like(q), torch.zeros(2, 300, device='cuda')\n"
        "st = torch.zeros(4, dtype=torch.int32, device='cuda'); p = dt.sparse_params(q, k, k, O, 64, 4)\n"
        "qm, km = torch.zeros(2, 3, 64, device='cuda'), torch.zeros(2, 4, 64, device='cuda')\n"
        "n, m = dt.norm_rope_params(q, norm=False), dt.norm_rope_params(k=k, norm=False)\n"
        "s = dt.select_params(2, 2, 3, 4, 64, 4); c = torch.zeros(2, 3, dtype=torch.int32, device='cuda')\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    dt.dt_qk_norm_rope(n, q, None, None, None, None, None, None, None, None, qm)\n"
        "    dt.dt_qk_norm_rope(m, None, k, None, None, None, None, None, None, None, None, km)\n"
        "    dt.dt_block_select(s, qm, km, idx, c)\n"
        "    dt.dt_attn_block_sparse(p, q, k, k, idx, c, O, L, st)\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "ref = torch.softmax(q.float() @ k.float().transpose(1, 2) / 8, -1) @ k.float()\n"
        "assert int(st[0]) == 0 and float((O.float() - ref).abs().max()) < 0.01\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("H", [2, 80])
def test_attention_rows_outside_the_lists_are_not_read(block, H):
    """Infinities and NaN in every key and value row that no list names change nothing."""
    g = gen(23)
    Sq, Sk, D, cap = 260, 1111, 64, 5
    q, k, v = randn(g, H, Sq, D, dtype=BF), randn(g, 1, Sk, D, dtype=BF), randn(g, 1, Sk, D, dtype=BF)
    idx, count = lists_for(g, H, Sq, Sk, block, cap, cap)
    odd = torch.arange(-(-Sk // block), device="cuda") % 2 == 1
    idx = (idx // 2 * 2).contiguous()                 # even blocks alone, some of them twice
    O, L, _ = attend(q, k, v, idx, count, block)
    rows = odd.repeat_interleave(block)[:Sk]
    k[:, rows], v[:, rows] = math.nan, math.inf
    O2, L2, st = attend(q, k, v, idx, count, block)
    assert st == 0 and torch.equal(O, O2) and torch.equal(L, L2)
    check_attention(q, torch.nan_to_num(k, 0.0), torch.where(rows[:, None], 0.0, v.float()).to(BF), idx, count, block, O, L)


def test_attention_masked_logits_of_minus_infinity():
    """Keys whose logit is -infinity weigh nothing; rows with no other key are empty."""
    H, Sq, Sk, D = 1, 130, 256, 64
    g = gen(29)
    q, k, v = randn(g, H, Sq, D, dtype=BF).abs(), randn(g, H, Sk, D, dtype=BF), randn(g, H, Sk, D, dtype=BF)
    k[:, :128] = 0
    k[:, :128, 0] = -math.inf
    idx = torch.tensor([[[0, 1], [0, 3]]], dtype=torch.int32, device="cuda")
    count = torch.tensor([[2, 2]], dtype=torch.int32, device="cuda")
    O, L, st = attend(q, k, v, idx, count, 64)
    assert st == 0 and bool((O[:, :128] == 0).all()) and bool(torch.isneginf(L[:, :128]).all())
    only = torch.tensor([[[3, 3], [3, 3]]], dtype=torch.int32, device="cuda")
    kf = torch.where(torch.isinf(k), torch.zeros_like(k), k)
    ref = sp.block_sparse_attention(np64(q), np64(kf), np64(v), only.cpu().numpy(), np.array([[1, 1]]), 64)
    within(O[:, 128:], ref[0][:, 128:], 2.0 ** -6 * (1 + ref[2][:, 128:]), "O")
    # a NaN value that a row attends shows in that row's block alone
    v[0, 200] = math.nan
    O, L, _ = attend(q, k, v, idx, count, 64)
    assert bool(torch.isfinite(O[:, :128]).all()) and bool(torch.isnan(O[:, 128:]).all())


def test_attention_bad_lists_are_reported_and_read_nothing():
    g = gen(31)
    H, Sq, Sk, D = 2, 300, 500, 72
    q, k, v = randn(g, H, Sq, D, dtype=BF), randn(g, H, Sk, D, dtype=BF), randn(g, H, Sk, D, dtype=BF)
    for block, nk in ((64, 8), (128, 4)):
        idx = torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda").expand(H, 3, 3).contiguous()
        count = torch.full((H, 3), 3, dtype=torch.int32, device="cuda")
        good = attend(q, k, v, idx, count, block)
        assert good[2] == 0
        for bad in (-1, nk, 2 ** 31 - 1, -2 ** 31):
            wrong = idx.clone()
            wrong[1, 1, 1] = bad
            O, L, st = attend(q, k, v, wrong, count, block)
            assert st == dt.DT_ERR_INVALID
            assert torch.equal(O[0], good[0][0]) and torch.equal(O[1, :128], good[0][1, :128])
            check_attention(q, k, v, wrong, count, block, O, L)
        for n, same in ((4, 3), (-1, 0), (2 ** 31 - 1, 3), (-2 ** 31, 0)):
            c = count.clone()
            c[0, 2] = n
            O, L, st = attend(q, k, v, idx, c, block)
            assert st == dt.DT_ERR_INVALID
            c[0, 2] = same
            O2, L2, st = attend(q, k, v, idx, c, block)
            assert st == 0 and torch.equal(O, O2) and torch.equal(L, L2)


def test_attention_empty_lists_no_counts_no_keys():
    g = gen(37)
    q, k, v = randn(g, 2, 140, 64, dtype=BF), randn(g, 2, 256, 64, dtype=BF), randn(g, 2, 256, 64, dtype=BF)
    idx = torch.zeros(2, 2, 0, dtype=torch.int32, device="cuda")
    for kk, vv, i, c in ((k, v, idx, None), (k[:, :0], v[:, :0], idx, None),
                         (k[:, :0], v[:, :0], idx.new_zeros(2, 2, 3), torch.zeros(2, 2, dtype=torch.int32, device="cuda"))):
        O, L, st = attend(q, kk, vv, i, c, 64)
        assert st == 0 and bool((O == 0).all()) and bool(torch.isneginf(L).all())
    full = torch.arange(4, dtype=torch.int32, device="cuda").expand(2, 2, 4).contiguous()
    O, L, st = attend(q, k, v, full, None, 64)        # no counts: every entry
    assert st == 0
    check_attention(q, k, v, full, torch.full((2, 2), 4, dtype=torch.int32), 64, O, L)


def test_attention_no_keys_with_dense_strides():
    """Dense strides {Sk * D, D} of no keys are {0, D}: they describe nothing, and refuse nothing."""
    H, Sq, D = 4, 140, 64
    q = randn(gen(38), H, Sq, D, dtype=BF)
    O, L = torch.full_like(q, 9.0), torch.full((H, Sq), 9.0, device="cuda")
    idx, count = torch.zeros(H, 2, 3, dtype=torch.int32, device="cuda"), torch.zeros(H, 2, dtype=torch.int32, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    dense = dt.Strides(Sq * D, D)
    p = dt.SparseParams(H, 2, Sq, 0, D, 64, 3, dt.DT_TYPE_BF16, dt.DT_TYPE_BF16, dense, dt.Strides(0, D), dt.Strides(0, D), dense)
    res = dt.load().dt_attn_block_sparse(ctypes.byref(p), q.data_ptr(), None, None, idx.data_ptr(), count.data_ptr(),
                                         O.data_ptr(), L.data_ptr(), st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert res == dt.DT_OK and int(st[0]) == 0
    assert bool((O == 0).all()) and bool(torch.isneginf(L).all())


def test_attention_strides_past_32_bits():
    """K and V heads and rows more than 2^31 elements apart."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = gen(41)
    D, far = 64, (1 << 31) + 64
    buf = torch.empty(far * 2 + 4096 * D, dtype=BF, device="cuda")
    k = buf.as_strided((2, 300, D), (far, D, 1))
    v = buf.as_strided((2, 300, D), (far, D, 1), 1000 * D)
    O = buf.as_strided((2, 140, D), (far, D, 1), 2000 * D)
    k.copy_(randn(g, 2, 300, D, dtype=BF))
    v.copy_(randn(g, 2, 300, D, dtype=BF))
    q = randn(g, 2, 140, D, dtype=BF)
    idx, count = lists_for(g, 2, 140, 300, 64, 4, 4)
    out, L, st = attend(q, k, v, idx, count, 64, o=O)
    assert st == 0
    check_attention(q, k, v, idx, count, 64, out, L)
    rows = torch.empty(far + 64, dtype=BF, device="cuda").as_strided((1, 2, D), (D, far, 1))
    rows.copy_(randn(g, 1, 2, D, dtype=BF))
    one = torch.zeros(1, 2, 1, dtype=torch.int32, device="cuda")
    out, L, st = attend(q[:1], rows, rows, one, None, 64)
    check_attention(q[:1], rows, rows, one, torch.ones(1, 2, dtype=torch.int32), 64, out, L)


def test_attention_fp32_states_compose_with_state_merge():
    """States of disjoint lists, merged, equal the state of their union."""
    g = gen(43)
    H, Sq, Sk, D = 3, 200, 640, 128
    q, k, v = randn(g, H, Sq, D, dtype=BF), randn(g, H, Sk, D, dtype=BF), randn(g, H, Sk, D, dtype=BF)
    perm = torch.rand(H, 2, 10, generator=g, device="cuda").argsort(-1).to(torch.int32)
    O_in, L_in = torch.empty(2, H, Sq, D, device="cuda"), torch.empty(2, H, Sq, device="cuda")
    for n, part in enumerate((perm[..., :4], perm[..., 4:])):
        O, L, st = attend(q, k, v, part.contiguous(), None, 64, oty=F32)
        O_in[n], L_in[n] = O, L
        check_attention(q, k, v, part, torch.full((H, 2), part.shape[-1], dtype=torch.int32), 64, O, L)
    O, L = torch.empty(H, Sq, D, device="cuda"), torch.empty(H, Sq, device="cuda")
    dt.dt_state_merge(2, H, Sq, D, O_in, L_in, O, L)
    check_attention(q, k, v, perm, torch.full((H, 2), 10, dtype=torch.int32), 64, O, L)


@pytest.mark.parametrize("H,Sq,Sk,cap", [(40, 1, 4096, 32), (8, 1024, 1024, 8)])
def test_attention_captured_replayed_on_other_streams_and_repeatable(H, Sq, Sk, cap):
    g = gen(47)
    D = 128
    q, k, v = randn(g, H, Sq, D, dtype=BF), randn(g, H, Sk, D, dtype=BF), randn(g, H, Sk, D, dtype=BF)
    idx, count = lists_for(g, H, Sq, Sk, 64, cap, RAGGED(cap))
    want_o, want_l, _ = attend(q, k, v, idx, count, 64)
    for _ in range(3):
        O, L, _ = attend(q, k, v, idx, count, 64)
        assert torch.equal(O, want_o) and torch.equal(L, want_l)
    # two calls at once on two streams, and two captured graphs replayed together
    outs = [(torch.empty_like(q), torch.empty(H, Sq, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"))
            for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    p = dt.sparse_params(q, k, v, outs[0][0], 64, cap)
    torch.cuda.synchronize()
    for s, (O, L, st) in zip(streams, outs):
        dt.dt_attn_block_sparse(p, q, k, v, idx, count, O, L, st, s)
    torch.cuda.synchronize()
    for O, L, st in outs:
        assert torch.equal(O, want_o) and torch.equal(L, want_l) and int(st[0]) == 0
    graphs = []
    for s, (O, L, st) in zip(streams, outs):
        O.zero_()
        L.zero_()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            dt.dt_attn_block_sparse(p, q, k, v, idx, count, O, L, st)
        graphs.append(gr)
    for _ in range(2):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for O, L, st in outs:
        assert torch.equal(O, want_o) and torch.equal(L, want_l) and int(st[0]) == 0


@pytest.mark.parametrize("H,Sq", [(4, 1024), (2, 1)])
def test_attention_wait_limit_reports_timeout_and_context_survives(H, Sq):
    g = gen(53)
    q, k, v = randn(g, H, Sq, 72, dtype=BF), randn(g, H, 1024, 72, dtype=BF), randn(g, H, 1024, 72, dtype=BF)
    idx, count = lists_for(g, H, Sq, 1024, 64, 16, 16)
    dt.dt_set_wait_limit_ns(0)
    try:
        _, _, st = attend(q, k, v, idx, count, 64)
    finally:
        dt.dt_set_wait_limit_ns(2_000_000_000)
    assert st == dt.DT_ERR_TIMEOUT
    O, L, st = attend(q, k, v, idx, count, 64)
    assert st == 0
    check_attention(q, k, v, idx, count, 64, O, L)


@pytest.mark.parametrize("ty", [BF, FP])
@pytest.mark.parametrize("H", [1, 80])
@pytest.mark.parametrize("heavy", [0, 33_000, 65_535])
def test_attention_many_light_keys_keep_their_weight(ty, H, heavy):
    """One key with nearly all the weight and 65,535 of a weight near 2^-25.4 each, below half of fp16's least step,
    which together are 1.5e-3 of a row."""
    D, Sk = 64, 65_536
    q = torch.zeros(H, 1, D, dtype=ty, device="cuda")
    k, v = torch.zeros(1, Sk, D, dtype=ty, device="cuda"), torch.ones(1, Sk, D, dtype=ty, device="cuda")
    q[..., 0], k[..., 0] = 8.0, -17.625
    k[0, heavy, 0], v[0, heavy] = 0.0, 0.0
    idx = torch.arange(Sk // 64, dtype=torch.int32, device="cuda").expand(H, 1, -1).contiguous()
    for oty in (ty, F32):
        O, L, st = attend(q, k, v, idx, None, 64, oty=oty)
        assert st == 0
        n, w = Sk - 1, math.exp(-17.625)
        ref = n * w / (1 + n * w)
        # logits are exact; ex2 and the weights' sum as in check_attention.  A rounded weight is off by half a step:
        # 2^-8 or 2^-11 of it, or, below fp16's normal range, 2^-25 of a scale on which the heaviest weight is at
        # least 2^7
        e = 2.0 ** -22 + Sk * 64 * 2.0 ** -24 / 32
        o = ref * (HALF[ty] + 2 * e) + TINY[ty] * 2.0 ** -7 * n
        bound = o + HALF[oty] * (ref + o) + TINY[oty]
        assert float((O.double() - ref).abs().max()) <= bound, (float(O.double().mean()), ref)
        assert float((L.double() - math.log1p(n * w)).abs().max()) <= e + 2.0 ** -22


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("H,S,D,dims,topk", [(2, 1000, 64, (24, 20, 20), 5), (16, 1024, 72, (36, 36), 8), (3, 2080, 128, (44, 42, 42), 9)])
def test_session_from_projection_to_sparse_output(H, S, D, dims, topk):
    """Projection -> norm, rotation, means -> lists -> attention, each stage against the oracle on the stage's
    own inputs; then the same through set_inputs, and a partition step afterwards as if nothing had been."""
    g = gen(59)
    side = 1 + int(S ** (1 / len(dims)))
    pos = torch.stack(torch.unravel_index(torch.arange(S, device="cuda"), (side + S,) + (side,) * (len(dims) - 1))).int()
    table = torch.empty(S, D // 2, 2, device="cuda")
    dt.dt_rope_table(dt.rope_params(S, dims), pos.contiguous(), table)
    qkv = randn(g, S, 3 * H * D, dtype=BF)
    wq, wk = 1 + 0.1 * randn(g, D), 1 + 0.1 * randn(g, D)
    sess = Session(H, S, D, P=4)
    sess.set_projection(qkv, wq, wk, table)
    x = np64(qkv).reshape(S, 3, H, D).transpose(1, 2, 0, 3)
    for i, (out, w) in enumerate(((sess.Q, wq), (sess.K, wk))):
        y, mag = sp.norm_rope(x[i], np64(w), sp.rope_table(pos.cpu().numpy(), dims)[0])
        within(out, y, 2.0 ** -18 * mag + HALF[BF] * 1.001 * np.abs(y), "QK"[i])
    assert torch.equal(sess.V, qkv.view(S, 3, H, D)[:, 2].transpose(0, 1))
    sess.step_sparse(topk, keep_first=1, margin=3.0, remeasure=False)
    sess.check()
    ref = sp.block_select(np64(sess.q_mean), np64(sess.k_mean), topk, 1, 0, 3.0)
    np.testing.assert_array_equal(sess.lists[0].cpu().numpy(), ref[0])
    np.testing.assert_array_equal(sess.lists[1].cpu().numpy(), ref[1])
    check_attention(sess.Q, sess.K, sess.V, *sess.lists, 64, sess.O, sess.L)
    # inputs set directly: the means are taken from them
    other = Session(H, S, D, P=4)
    other.set_inputs(sess.Q, sess.K, sess.V)
    with pytest.raises(ValueError):
        other.step_sparse(topk, remeasure=False)
    other.step_sparse(topk, k_block=128)
    other.check()
    within(other.q_mean, sp.block_means(np64(sess.Q), 128), 2.0 ** -17 * sp.block_means(np.abs(np64(sess.Q)), 128), "q_mean")
    check_attention(other.Q, other.K, other.V, *other.lists, 128, other.O, other.L)
    # every block selected is the partition step's full attention
    other.step_sparse(-(-S // 64))
    full_o, full_l = other.O.clone(), other.L.clone()
    other.step(1)
    other.check()
    assert float((other.O.float() - full_o.float()).abs().max()) <= 2e-2 and float((other.L - full_l).abs().max()) <= 1e-3
    ref_o, ref_l = orc.attention_state(np64(sess.Q[0, :5]), np64(sess.K[0]), np64(sess.V[0]), orc.softmax_scale(D))
    assert np.abs(np64(full_o[0, :5]) - ref_o).max() <= 2e-2 and np.abs(np64(full_l[0, :5]) - ref_l).max() <= 1e-3


def test_session_sparse_step_captured_in_a_graph():
    g = gen(61)
    H, S, D = 4, 1500, 128
    qkv = randn(g, S, 3 * H * D, dtype=BF)
    sess = Session(H, S, D, P=2, cache=False)
    sess.set_projection(qkv)
    sess.step_sparse(6, remeasure=False)
    want = sess.O.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sess.set_projection(qkv)
        sess.step_sparse(6, remeasure=False)
    sess.O.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(sess.O, want)
    qkv.mul_(-1.0)                                    # new inputs, same graph
    graph.replay()
    sess.check()
    sess2 = Session(H, S, D, P=2, cache=False)
    sess2.set_projection(qkv)
    sess2.step_sparse(6, remeasure=False)
    assert torch.equal(sess.O, sess2.O) and torch.equal(sess.lists[0], sess2.lists[0])


def test_session_sparse_steps_of_several_sizes_beside_a_captured_one():
    """Other topk and k_block in between leave a captured sparse step's buffers alone."""
    g = gen(67)
    H, S, D = 3, 900, 64
    qkv = randn(g, S, 3 * H * D, dtype=BF)
    sess = Session(H, S, D, P=2, cache=False)
    sess.set_projection(qkv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sess.step_sparse(5)
    graph.replay()
    torch.cuda.synchronize()
    want_o, want_l = sess.O.clone(), sess.lists[0].clone()
    lists = sess.lists
    sess.step_sparse(3, k_block=128)
    with pytest.raises(ValueError):
        sess.step_sparse(3, remeasure=False)          # the means at hand are of 128-row blocks
    sess.step_sparse(4, remeasure=False, k_block=128)
    sess.set_inputs(sess.Q.clone(), sess.K.clone(), sess.V.clone())
    with pytest.raises(ValueError):
        sess.step_sparse(4, remeasure=False, k_block=128)
    with pytest.raises(ValueError):
        sess.step_sparse(4, k_block=96)
    with pytest.raises(ValueError):
        sess.set_projection(qkv[:, :-8])
    sess.O.zero_()
    graph.replay()
    sess.check()
    assert torch.equal(sess.O, want_o) and torch.equal(lists[0], want_l)


@pytest.mark.parametrize("raw", [False, True])
def test_session_buffers_of_a_first_call_belong_to_its_stream(raw):
    """The first set_projection and step_sparse of a size, on a stream of their own while the current stream is busy:
    memory freed on the current stream, which its pending work still reads, is not handed to them."""
    g = gen(71)
    H, S, D, topk = 4, 1000, 64, 5
    qkv = randn(g, S, 3 * H * D, dtype=BF)
    ref = Session(H, S, D, P=2, cache=False)
    ref.set_projection(qkv)
    ref.step_sparse(topk, remeasure=False)
    sess, side = Session(H, S, D, P=2, cache=False), torch.cuda.Stream()
    torch.cuda.synchronize()
    nq, nk = -(-S // 128), -(-S // 64)
    old = [torch.full((n,), 5.0, device="cuda") for n in (H * nq * D, H * nk * D, H * nq * topk, H * nq)]
    seen = [torch.empty_like(t) for t in old]
    torch.cuda._sleep(100_000_000)                    # the copies below stay pending for tens of milliseconds
    for t, u in zip(old, seen):
        u.copy_(t)
    del old, t
    stream = side.cuda_stream if raw else side
    sess.set_projection(qkv, stream=stream)
    sess.step_sparse(topk, remeasure=False, stream=stream)
    torch.cuda.synchronize()
    assert all(bool((u == 5.0).all()) for u in seen)
    assert torch.equal(sess.O, ref.O) and torch.equal(sess.L, ref.L) and torch.equal(sess.lists[0], ref.lists[0])


def test_session_lists_of_two_block_sizes_and_one_length():
    """The same topk with both block sizes: neither step overwrites the other's lists, captured or not."""
    g = gen(73)
    H, S, D, topk = 2, 1000, 64, 4
    sess = Session(H, S, D, P=2, cache=False)
    sess.set_inputs(*(randn(g, H, S, D, dtype=BF) for _ in range(3)))
    sess.step_sparse(topk, k_block=64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sess.step_sparse(topk, k_block=64)
    lists = sess.lists
    graph.replay()
    want = [t.clone() for t in lists]
    sess.step_sparse(topk, k_block=128)
    other, want_other = sess.lists, [t.clone() for t in sess.lists]
    assert all(torch.equal(a, b) for a, b in zip(lists, want))
    graph.replay()
    sess.check()
    assert all(torch.equal(a, b) for a, b in zip(other, want_other))
    assert all(torch.equal(a, b) for a, b in zip(lists, want))


def test_session_block_means_of_captured_projections():
    """A captured set_projection measures nothing until it is replayed, and a replay is not seen by the session:
    remeasure=False takes the means that ran last or were declared."""
    g = gen(79)
    H, S, D = 2, 900, 64
    qkv = randn(g, S, 3 * H * D, dtype=BF)
    ref = Session(H, S, D, P=2, cache=False)
    ref.set_projection(qkv)
    ref.step_sparse(5, remeasure=False)
    torch.cuda.synchronize()
    sess = Session(H, S, D, P=2, cache=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sess.set_projection(qkv)
        sess.step_sparse(5, remeasure=False)          # what the replay measures before it
    with pytest.raises(ValueError):
        sess.step_sparse(5, remeasure=False)          # nothing has run
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(sess.O, ref.O)
    sess.declare_means(64)
    sess.O.zero_()
    sess.step_sparse(5, remeasure=False)
    sess.check()
    assert torch.equal(sess.O, ref.O) and torch.equal(sess.lists[0], ref.lists[0])
    # a replay after an eager projection with the other block size, and after inputs set directly
    sess.set_projection(-2 * qkv, k_block=128)
    sess.step_sparse(5, remeasure=False, k_block=128)
    graph.replay()
    sess.declare_means(64)
    with pytest.raises(ValueError):
        sess.step_sparse(5, remeasure=False, k_block=128)
    sess.step_sparse(5, remeasure=False)
    sess.check()
    assert torch.equal(sess.O, ref.O)
    sess.set_inputs(ref.Q, ref.K, ref.V)
    with pytest.raises(ValueError):
        sess.step_sparse(5, remeasure=False)
    sess.set_projection(qkv)
    sess.declare_means(None)                          # Q or K changed behind the session's back
    with pytest.raises(ValueError):
        sess.step_sparse(5, remeasure=False)
    # a captured projection with another block size leaves no eager claim behind
    sess.set_projection(qkv)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        sess.set_projection(qkv, k_block=128)
    for k_block in (64, 128):
        with pytest.raises(ValueError):
            sess.step_sparse(5, remeasure=False, k_block=k_block)
    for bad in (96, 0):
        with pytest.raises(ValueError):
            sess.declare_means(bad)
    with pytest.raises(ValueError):
        Session(H, S, D, P=2, cache=False).declare_means(64)      # never measured


@pytest.mark.parametrize("device", ["cuda", "cuda:0", torch.device("cuda", 0)])
def test_session_keeps_the_device_it_was_made_on(device):
    """"cuda" means the device that is current now, also for buffers allocated by later calls."""
    with torch.cuda.device(0):
        sess = Session(2, 300, 64, P=2, device=device, cache=False)
    assert sess.device == sess.Q.device == torch.device("cuda", 0)
    sess.set_inputs(*(randn(gen(97), 2, 300, 64, dtype=BF) for _ in range(3)))
    sess.step_sparse(2)
    sess.check()
    assert sess.q_mean.device == sess.lists[0].device == sess.device


# ------------------------------------------------------------------ fp32 states
def attend_f32(q, k, v, idx, count, block, token_major):
    """O as fp32, dense or token-major (head-major view of [Sq][H][D])."""
    H, Sq, D = q.shape
    o = torch.full((Sq, H, D), 9.0, device="cuda").transpose(0, 1) if token_major else None
    O, L, st = attend(q, k, v, idx, count, block, oty=F32, o=o)
    assert st == 0
    check_attention(q, k, v, idx, count, block, O, L)


@pytest.mark.parametrize("ty", [BF, FP])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("H,Hkv,Sq,Sk,block,cap", [(1, 1, 1, 1, 64, 1), (2, 1, 129, 200, 128, 2), (4, 2, 300, 1000, 64, 7),
                                                   (3, 3, 257, 777, 128, 5), (2, 1, 17, 4100, 64, 65)])
def test_fp32_states_sizes(ty, D, H, Hkv, Sq, Sk, block, cap):
    g = gen(Sq + Sk + 1)
    q, k, v = randn(g, H, Sq, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty)
    for counts, token_major in ((cap, False), (RAGGED(cap), True), (0, True)):
        idx, count = lists_for(g, H, Sq, Sk, block, cap, counts)
        attend_f32(q, k, v, idx, count, block, token_major)


@pytest.mark.parametrize("ty", [BF, FP])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("H,Sq,cap", [(1, 1, 33), (5, 130, 30), (20, 100, 64), (74, 3, 8)])
def test_fp32_states_of_lists_split_over_a_cluster(ty, D, H, Sq, cap):
    g = gen(83)
    block, Sk = 64, 64 * 64
    q, k, v = randn(g, H, Sq, D, dtype=ty), randn(g, 1, Sk, D, dtype=ty), randn(g, 1, Sk, D, dtype=ty)
    for counts, token_major in ((cap, True), (RAGGED(cap), False), (1, False)):
        idx, count = lists_for(g, H, Sq, Sk, block, cap, counts)
        attend_f32(q, k, v, idx, count, block, token_major)


@pytest.mark.parametrize("ty", [BF, FP])
@pytest.mark.parametrize("H,Hkv,Sq,D,block", [(40, 40, 600, 128, 64), (160, 20, 128, 64, 128), (30, 30, 700, 72, 64)])
def test_fp32_states_of_many_items_per_cta(ty, H, Hkv, Sq, D, block):
    g = gen(89)
    Sk, cap = 1500, 9
    q, k, v = randn(g, H, Sq, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty), randn(g, Hkv, Sk, D, dtype=ty)
    idx, count = lists_for(g, H, Sq, Sk, block, cap, RAGGED(cap))
    for token_major in (False, True):
        attend_f32(q, k, v, idx, count, block, token_major)


# ------------------------------------------------------------------ far rotations
TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")


def rope_table_60_digits(pos, dims, base):
    """(cos, sin) with the turns and their reduction in 60 digits; off by less than 2^-49."""
    with localcontext() as ctx:
        ctx.prec = 60
        cols = []
        for p, dim in zip(pos, dims):
            for j in range(dim // 2):
                turn = Decimal(base) ** (Decimal(-2 * j) / dim) / TWO_PI
                cols.append([float(x - x.to_integral_value()) for x in (int(v) * turn for v in p)])
    angle = 2 * np.pi * np.array(cols).T
    return np.stack([np.cos(angle), np.sin(angle)], axis=-1)


def test_the_60_digit_oracle_is_the_tables_formula():
    pos = np.array([[0, 1, -7, 1000], [3, -2, 11, 0]])
    ref, _ = sp.rope_table(pos, (12, 8), 10000.0)
    np.testing.assert_allclose(rope_table_60_digits(pos, (12, 8), 10000.0), ref, atol=1e-12)


@pytest.mark.parametrize("axes,base", [((128,), 10000.0), ((256,), 2.0), ((44, 42, 42), 1e6), ((6, 10), 10000.0),
                                       ((64, 2), 1.0), ((72,), 500000.0), ((256,), 1.01), ((40, 4), 1e300)])
def test_rope_table_far_positions(axes, base):
    """Positions to both ends of int32, against angles reduced in 60 digits.

    A frequency is held within 2^-58 of a turn: truncation takes 2^-64, and at most 127 extended-precision products
    with a power that is itself within two units leave 0.16 e^-z (3 * 127 + z + 2) 2^-64 < 2^-58, z = the frequency's
    negative logarithm.  The reduced angle's rounding takes 2 pi 2^-28, the polynomials and their evaluation at most
    three roundings of values below 1: 2^-22 in all."""
    g = np.random.Generator(np.random.PCG64(len(axes)))
    far = [-2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 30 - 12345, 2 ** 30 + 54321, -1, 0, 1, -131071, 1 << 20]
    pos = np.array([np.concatenate([np.roll(far, a), g.integers(-2 ** 31, 2 ** 31, 20)]) for a in range(len(axes))])
    table = torch.empty(pos.shape[1], sum(axes) // 2, 2, device="cuda")
    dt.dt_rope_table(dt.rope_params(pos.shape[1], axes, base), torch.from_numpy(pos.astype(np.int32)).cuda(), table)
    axis = np.repeat(np.arange(len(axes)), np.array(axes) // 2)
    bound = 2.0 ** -22 + 2 * np.pi * 2.0 ** -58 * np.abs(pos[axis].T.astype(np.float64))
    within(table, rope_table_60_digits(pos, axes, base), bound[..., None], "table")
