"""Block-sparse attention and the passes in front of it, without a GPU: struct
layouts, argument validation of the C entry points and of the binding.  Every
call here is refused, or has nothing to do, before any CUDA call."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import partitioned_attention_state_b200 as dt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20            # an aligned address that no refused call touches


@pytest.mark.skipif(not shutil.which("gcc"), reason="no C compiler")
def test_structs_have_the_headers_layout(tmp_path):
    structs = {"dt_strides": dt.Strides, "dt_rope_params": dt.RopeParams, "dt_norm_rope_params": dt.NormRopeParams,
               "dt_select_params": dt.SelectParams, "dt_sparse_params": dt.SparseParams}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "dt.h"', "int main(void) {"]
    for c, s in structs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{n} %zu\\n", offsetof({c}, {n}));' for n, _ in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    want = {}
    for c, s in structs.items():
        want[c] = ctypes.sizeof(s)
        want |= {f"{c}.{n}": getattr(s, n).offset for n, _ in s._fields_}
    assert {k: int(v) for k, v in (line.split() for line in out.splitlines())} == want


# ------------------------------------------------------------------ rope table
def rope(S=4, axes=(8, 8), base=10000.0, pos=P, table=P, **over):
    p = dt.rope_params(S, axes, base)
    for k, v in over.items():
        setattr(p, k, v)
    return dt.load().dt_rope_table(ctypes.byref(p), pos, table, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(axes=(7,)), dict(axes=(0,)), dict(axes=(-2,)), dict(axes=(200, 58)),
                                dict(base=0.0), dict(base=-1.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(base=0.99), dict(S=(1 << 30) + 1),
                                dict(pos=None), dict(table=None), dict(n_axes=0), dict(n_axes=5)])
def test_rope_table_refuses(kw):
    assert rope(**kw) == dt.DT_ERR_INVALID


def test_rope_table_alignment_and_nothing_to_do():
    assert rope(pos=P + 4) == dt.DT_ERR_UNSUPPORTED
    assert rope(table=P + 8) == dt.DT_ERR_UNSUPPORTED
    assert rope(S=0, pos=None, table=None) == dt.DT_OK
    assert dt.load().dt_rope_table(None, P, P, None) == dt.DT_ERR_INVALID


# ------------------------------------------------------------------ norm + rotation
NR = dict(S=10, D=64, H=2, Hkv=2, rot=64, pairing=0, in_type=0, out_type=0, norm=1, q_block=128, k_block=64, eps=1e-6)
NAMES = ("q", "k", "v", "wq", "wk", "table", "Q", "K", "V", "q_mean", "k_mean")


def norm_rope(ptrs=None, strides=None, **over):
    p = dt.NormRopeParams(**{**NR, **over})
    for n in ("q_in", "k_in", "v_in", "q_out", "k_out", "v_out"):
        setattr(p, n, (strides or {}).get(n, dt.Strides(p.S * p.D, p.D)))
    args = {**{n: P for n in NAMES}, **(ptrs or {})}
    return dt.load().dt_qk_norm_rope(ctypes.byref(p), *[args[n] for n in NAMES], None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(S=(1 << 30) + 1), dict(D=0), dict(D=60), dict(D=136), dict(H=-1),
                                dict(Hkv=-1), dict(rot=-8), dict(rot=4), dict(rot=72), dict(pairing=2), dict(in_type=3),
                                dict(out_type=-1), dict(norm=2), dict(q_block=96), dict(k_block=0), dict(eps=-1e-6),
                                dict(eps=float("nan"))])
def test_norm_rope_refuses_parameters(kw):
    assert norm_rope(**kw) == dt.DT_ERR_INVALID


@pytest.mark.parametrize("ptrs", [dict(q=None), dict(k=None), dict(v=None), dict(V=None), dict(table=None),
                                  dict(Q=None, q_mean=None), dict(K=None, k_mean=None), dict(q=None, Q=None)])
def test_norm_rope_refuses_parts_that_do_not_match(ptrs):
    assert norm_rope(ptrs) == dt.DT_ERR_INVALID


def test_norm_rope_types_alignment_strides():
    assert norm_rope(out_type=1) == dt.DT_ERR_UNSUPPORTED                       # bf16 in, fp16 out
    assert norm_rope(in_type=1, out_type=2) == dt.DT_ERR_UNSUPPORTED
    for n in NAMES:
        assert norm_rope({n: P + 8}) == dt.DT_ERR_UNSUPPORTED, n
    for n in ("q_in", "k_in", "v_in", "q_out", "k_out", "v_out"):
        assert norm_rope(strides={n: dt.Strides(640, 60)}) == dt.DT_ERR_UNSUPPORTED, n
        assert norm_rope(strides={n: dt.Strides(636, 64)}) == dt.DT_ERR_UNSUPPORTED, n
        assert norm_rope(strides={n: dt.Strides(640, -64)}) == dt.DT_ERR_INVALID, n
    assert norm_rope(S=0) == dt.DT_OK
    none = {n: None for n in NAMES}
    assert norm_rope(none) == dt.DT_OK                                          # no part at all


def test_norm_rope_in_place_needs_the_same_layout():
    one = {**{n: None for n in NAMES}, "q": P, "Q": P, "wq": P, "table": P}
    assert norm_rope(one, in_type=2, out_type=0) == dt.DT_ERR_INVALID
    assert norm_rope(one, strides=dict(q_out=dt.Strides(640, 128))) == dt.DT_ERR_INVALID
    assert norm_rope(one, strides=dict(q_out=dt.Strides(1280, 64))) == dt.DT_ERR_INVALID


def test_norm_rope_output_rows_do_not_share_memory():
    """A stride of 0 broadcasts an input; as an output's it would have rows or heads overwrite one another."""
    for n in ("q_out", "k_out", "v_out"):
        assert norm_rope(strides={n: dt.Strides(640, 0)}) == dt.DT_ERR_INVALID, n
        assert norm_rope(strides={n: dt.Strides(0, 64)}) == dt.DT_ERR_INVALID, n
    # in place on a broadcast input
    one = {**{n: None for n in NAMES}, "q": P, "Q": P, "wq": P, "table": P}
    for st in (dt.Strides(640, 0), dt.Strides(0, 64)):
        assert norm_rope(one, strides=dict(q_in=st, q_out=st)) == dt.DT_ERR_INVALID
    # nothing to write: no rows share memory
    apart = dict(Q=P + 4096, K=P + 8192, V=P + 12288)
    assert norm_rope(apart, S=0, strides={n: dt.Strides(0, 0) for n in ("q_out", "k_out", "v_out")}) == dt.DT_OK


# ------------------------------------------------------------------ selection
SEL = dict(H=4, Hkv=2, nq=3, nk=5, D=64, topk=2, keep_first=0, keep_last=0, margin=float("inf"))


def select(qm=P, km=P, idx=P, count=P, **over):
    p = dt.SelectParams(**{**SEL, **over})
    return dt.load().dt_block_select(ctypes.byref(p), qm, km, idx, count, None)


@pytest.mark.parametrize("kw", [dict(H=-1), dict(Hkv=0), dict(Hkv=3), dict(nq=-1), dict(nk=-1), dict(D=0), dict(D=66),
                                dict(D=132), dict(topk=0), dict(keep_first=-1), dict(keep_last=-1),
                                dict(keep_first=2, keep_last=1), dict(margin=-1.0), dict(margin=float("nan")),
                                dict(qm=None), dict(km=None), dict(idx=None), dict(count=None),
                                dict(H=1 << 16, Hkv=1, nq=1 << 15), dict(keep_first=2 ** 31 - 1, keep_last=2)])
def test_select_refuses(kw):
    assert select(**kw) == dt.DT_ERR_INVALID


def test_select_limits_and_nothing_to_do():
    assert select(nk=16385) == dt.DT_ERR_UNSUPPORTED
    for n in ("qm", "km", "idx", "count"):
        assert select(**{n: P + 4}) == dt.DT_ERR_UNSUPPORTED, n
    assert select(H=0) == dt.DT_OK
    assert select(nq=0, idx=None) == dt.DT_OK


@pytest.mark.parametrize("kw", [dict(topk=(1 << 30) + 1), dict(topk=2 ** 31 - 1), dict(H=1, Hkv=1, nq=(1 << 30) + 1),
                                dict(H=1, Hkv=1, nq=2 ** 31 - 1)])
def test_select_refuses_sizes_that_index_sums_would_pass(kw):
    assert select(**kw) == dt.DT_ERR_INVALID


# ------------------------------------------------------------------ attention
SP = dict(H=4, Hkv=2, Sq=100, Sk=200, D=64, k_block=64, cap=3, type=0, out_type=0)


def attend(ptrs=None, strides=None, **over):
    p = dt.SparseParams(**{**SP, **over})
    for n, rows in (("q", p.Sq), ("k", p.Sk), ("v", p.Sk), ("o", p.Sq)):
        setattr(p, n, (strides or {}).get(n, dt.Strides(max(rows, 1) * p.D, p.D)))
    names = ("Q", "K", "V", "idx", "count", "O", "L", "status")
    args = {**{n: P for n in names}, **(ptrs or {})}
    return dt.load().dt_attn_block_sparse(ctypes.byref(p), *[args[n] for n in names], None)


@pytest.mark.parametrize("kw", [dict(H=-1), dict(Hkv=0), dict(Hkv=3), dict(Sq=-1), dict(Sk=-1), dict(Sq=(1 << 30) + 1),
                                dict(Sk=(1 << 30) + 1), dict(cap=-1), dict(k_block=32), dict(k_block=0), dict(type=3),
                                dict(out_type=7), dict(H=1 << 24, Hkv=1, Sq=1 << 10)])
def test_attention_refuses_parameters(kw):
    assert attend(**kw) == dt.DT_ERR_INVALID


@pytest.mark.parametrize("cap", [(1 << 30) + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("k_block", [64, 128])
def test_attention_refuses_lists_that_index_sums_would_pass(cap, k_block):
    assert attend(cap=cap, k_block=k_block) == dt.DT_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(D=32), dict(D=80), dict(D=256), dict(type=2, out_type=2), dict(out_type=1)])
def test_attention_does_not_support(kw):
    assert attend(**kw) == dt.DT_ERR_UNSUPPORTED


@pytest.mark.parametrize("n", ["Q", "K", "V", "idx", "O", "L", "status"])
def test_attention_needs_its_buffers(n):
    assert attend({n: None}) == dt.DT_ERR_INVALID


def test_attention_alignment_strides_and_nothing_to_do():
    for n in ("Q", "K", "V", "idx", "count", "O", "L", "status"):
        assert attend({n: P + 4}) == dt.DT_ERR_UNSUPPORTED, n
    for n in ("q", "k", "v", "o"):
        assert attend(strides={n: dt.Strides(64 * 200, 68)}) == dt.DT_ERR_UNSUPPORTED, n
        assert attend(strides={n: dt.Strides(64 * 200 + 4, 64)}) == dt.DT_ERR_UNSUPPORTED, n
        assert attend(strides={n: dt.Strides(64 * 200, 0)}) == dt.DT_ERR_INVALID, n
        assert attend(strides={n: dt.Strides(-64 * 200, 64)}) == dt.DT_ERR_INVALID, n
        assert attend(strides={n: dt.Strides(1 << 39, 64)}) == dt.DT_ERR_INVALID, n
    assert attend({"count": None}, Sk=0) == dt.DT_ERR_INVALID
    assert attend(H=0, Hkv=0) == dt.DT_OK
    assert attend(Sq=0) == dt.DT_OK


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_tensors_that_do_not_fit():
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    Q, K = torch.zeros(4, 100, 64, dtype=bf), torch.zeros(2, 200, 64, dtype=bf)
    p = dt.sparse_params(Q, K, K, Q, 64, 3)
    idx, count = torch.zeros(4, 1, 3, dtype=i32), torch.zeros(4, 1, dtype=i32)
    L, st = torch.zeros(4, 100), torch.zeros(4, dtype=i32)
    good = dict(Q=Q, K=K, V=K, idx=idx, count=count, O=Q, L=L, d_status=st)
    bad = [dict(K=K[:, :199]), dict(V=K.half()), dict(O=Q.float()), dict(idx=idx.long()), dict(idx=idx[..., :2]),
           dict(count=count[:3]), dict(L=L.double()), dict(L=L.T), dict(Q=Q.transpose(1, 2)), dict(d_status=L)]
    for b in bad:
        with pytest.raises(ValueError):
            dt.dt_attn_block_sparse(p, **{**good, **b})
    with pytest.raises(ValueError, match="CUDA"):
        dt.dt_attn_block_sparse(p, **good)
    with pytest.raises(ValueError):
        dt.sparse_params(Q[..., ::2], K, K, Q)
    with pytest.raises(TypeError):
        dt.sparse_params(Q.double(), K, K, Q)

    s = dt.select_params(4, 2, 1, 4, 64, 3)
    good = dict(q_mean=torch.zeros(4, 1, 64), k_mean=torch.zeros(2, 4, 64), idx=idx, count=count)
    for b in [dict(q_mean=torch.zeros(4, 1, 64, dtype=bf)), dict(k_mean=torch.zeros(2, 3, 64)), dict(idx=idx[:, :, :2]),
              dict(count=count.long())]:
        with pytest.raises(ValueError):
            dt.dt_block_select(s, **{**good, **b})

    r = dt.rope_params(10, (8, 8))
    with pytest.raises(ValueError):
        dt.dt_rope_table(r, torch.zeros(1, 10, dtype=i32), torch.zeros(10, 8, 2))
    with pytest.raises(ValueError):
        dt.dt_rope_table(r, torch.zeros(2, 10, dtype=i32), torch.zeros(10, 4, 2))
    with pytest.raises(ValueError):
        dt.rope_params(10, (2,) * 5)

    n = dt.norm_rope_params(Q, K, None, Q, K, None, rot=64)
    args = dict(q=Q, k=K, v=None, wq=None, wk=None, table=torch.zeros(100, 32, 2), Q=Q, K=K, V=None)
    for b in [dict(K=K.float()), dict(table=torch.zeros(99, 32, 2)), dict(wq=torch.zeros(63)), dict(q=Q[:3]),
              dict(q_mean=torch.zeros(4, 2, 64))]:
        with pytest.raises(ValueError):
            dt.dt_qk_norm_rope(n, **{**args, **b})
    with pytest.raises(ValueError):
        dt.norm_rope_params()
