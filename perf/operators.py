"""The operators between a layer's projections and its attention output, as
plain torch and as the library's kernels.

A video or image transformer layer that attends sparsely runs four of them:

  rope     cos/sin table of the token positions (once per sequence geometry);
  norm     per-head RMS norm of queries and keys, position rotation, change
           from the projection's token-major layout to [head][token][D], and
           the block means of the results, in one pass;
  select   the key blocks each query block attends, by the scaled product of
           the block means;
  attend   attention of every query block over its selected key blocks only,
           giving the state (OUT, LSE).

``run`` computes one of them on what ``prepare`` made: with ``own`` false from
elementary torch operations, with ``own`` true through the library.
"""

import math

import numpy as np
import torch

own = False

QBLOCK = 128                       # query rows that share one list of key blocks
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NO_MARGIN = 1e9                    # select keeps the best topk, however far apart their scores are


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the angle table of a 32x32 patch grid, two axes sharing D = 72
        dict(name="rope_32x32", op="rope", S=1024, axes="36,36", grid="32,32", far=0),
        # the table of a 21x30x52 latent video, three axes sharing D = 128
        dict(name="rope_21x30x52", op="rope", S=32760, axes="44,42,42", grid="21,30,52", far=0),
        # one new token of a causal rollout, rotated far from the origin and put behind a long cache
        dict(name="norm_one_token", op="norm", S=1, H=40, Hkv=40, D=128, rot=128, halves=True, type="bf16", out="bf16",
             block=64, means=False),
        # a 32x32 image's layer, 16 heads of 72
        dict(name="norm_32x32_h16_d72", op="norm", S=1024, H=16, Hkv=16, D=72, rot=72, halves=False, type="bf16",
             out="bf16", block=64, means=True),
        # a video layer's whole sequence, 40 heads of 128, with the block means that select needs
        dict(name="norm_21x30x52_h40_d128", op="norm", S=32760, H=40, Hkv=40, D=128, rot=128, halves=False,
             type="bf16", out="bf16", block=64, means=True),
        # selection for a 32x32 image: a handful of blocks a head
        dict(name="select_32x32_h16", op="select", H=16, Hkv=16, nq=8, nk=16, D=72, topk=8, first=0, last=0,
             margin=NO_MARGIN),
        # selection for a video layer: an eighth of 512 blocks, the text blocks at the end always kept
        dict(name="select_video_h40", op="select", H=40, Hkv=40, nq=256, nk=512, D=128, topk=64, first=0, last=8,
             margin=4.0),
        # one new token over a long video's keys: memory-bound
        dict(name="attend_one_token", op="attend", H=40, Hkv=40, Sq=1, Sk=32760, D=128, block=64, cap=128, full=True,
             type="bf16"),
        # a 32x32 image at half the blocks: launch and latency bound
        dict(name="attend_32x32_h16_d72", op="attend", H=16, Hkv=16, Sq=1024, Sk=1024, D=72, block=64, cap=8, full=True,
             type="bf16"),
        # shared key heads, odd lengths, lists of every length from none
        dict(name="attend_shared_heads_ragged", op="attend", H=32, Hkv=8, Sq=1999, Sk=10007, D=64, block=128, cap=40,
             full=False, type="fp16"),
        # a 128x128 latent image, a quarter of the blocks
        dict(name="attend_128x128_h16_d72", op="attend", H=16, Hkv=16, Sq=16384, Sk=16384, D=72, block=64, cap=64,
             full=True, type="bf16"),
        # a video layer's sequence at an eighth of the blocks
        dict(name="attend_21x30x52_h40_d128", op="attend", H=40, Hkv=40, Sq=32760, Sk=32760, D=128, block=64, cap=64,
             full=True, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm", "select", "attend", "attend"])
    if op == "rope":
        n = rng.choice([1, 2, 3])
        grid = [max(1, _log(rng, 1, 32)) for _ in range(n)]
        return dict(op=op, S=math.prod(grid), axes=",".join(str(2 * rng.randint(4, 21)) for _ in range(n)),
                    grid=",".join(map(str, grid)), far=rng.choice([0, _log(rng, 1, 1 << 20)]))
    D = rng.choice([64, 72, 128])
    Hkv = rng.randint(1, 10)
    H = Hkv * rng.choice([1, 1, 2, 4])
    if op == "norm":
        return dict(op=op, S=_log(rng, 1, 32760), H=H, Hkv=Hkv, D=D, rot=8 * rng.randint(1, D // 8),
                    halves=rng.random() < 0.5, type=(t := rng.choice(["bf16", "fp16", "fp32"])),
                    out=rng.choice([t, "bf16"]), block=rng.choice([64, 128]), means=rng.random() < 0.7)
    if op == "select":
        nk = _log(rng, 16, 512)
        topk = rng.randint(6, max(6, nk // 2))
        return dict(op=op, H=H, Hkv=Hkv, nq=_log(rng, 1, 256), nk=nk, D=D, topk=topk,
                    first=rng.randint(0, 2), last=rng.randint(0, 2), margin=rng.choice([NO_MARGIN, 2.0, 5.0]))
    block = rng.choice([64, 128])
    Sq, Sk = rng.choice([(1, _log(rng, 1, 65536)), (n := _log(rng, 2, 32760), n),
                         (_log(rng, 2, 5000), _log(rng, 2, 32760))])
    nk = -(-Sk // block)
    cap = rng.randint(1, max(1, min(nk, 4096 // block)) if Sq > 512 else nk)
    return dict(op=op, H=H, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, block=block, cap=cap, full=rng.random() < 0.5,
                type=rng.choice(["bf16", "fp16"]))


def _counts(case):
    """Length of every list of an "attend" case, [H][query blocks]."""
    nq = -(-case["Sq"] // QBLOCK)
    h, q = np.meshgrid(np.arange(case["H"]), np.arange(nq), indexing="ij")
    if case["full"]:
        return np.full((case["H"], nq), case["cap"], np.int32)
    return ((7 * h + 13 * q + case["cap"] // 2 + 1) % (case["cap"] + 1)).astype(np.int32)


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dev = case["op"], "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if op == "rope":
        axes, grid = ([int(x) for x in case[k].split(",")] for k in ("axes", "grid"))
        # a sequence that starts anywhere on its first axis; positions are whole numbers
        start = case["far"] + int(torch.randint(0, 64, (1,), generator=g, device=dev))
        token = torch.arange(case["S"], device=dev)
        pos = torch.stack(torch.unravel_index(token, grid)).to(torch.int32)
        pos[0] += start
        return dict(case=case, axes=axes, pos=pos.contiguous(), table=torch.empty(case["S"], sum(axes) // 2, 2, device=dev))

    if op == "norm":
        S, H, Hkv, D, ty = case["S"], case["H"], case["Hkv"], case["D"], TYPES[case["type"]]
        x = (normal(S, H + 2 * Hkv, D) * (0.5 + normal(1, H + 2 * Hkv, 1).abs())).to(ty)   # the packed projection
        angle = torch.rand(S, case["rot"] // 2, generator=g, device=dev, dtype=torch.float64) * 2000 - 1000
        n = -(-S // QBLOCK), -(-S // case["block"])
        out = TYPES[case["out"]]
        return dict(case=case, x=x, wq=1 + 0.1 * normal(D), wk=1 + 0.1 * normal(D),
                    table=torch.stack([angle.cos(), angle.sin()], -1).float(),
                    Q=torch.empty(H, S, D, dtype=out, device=dev), K=torch.empty(Hkv, S, D, dtype=out, device=dev),
                    V=torch.empty(Hkv, S, D, dtype=out, device=dev),
                    qm=torch.empty(H, n[0], D, device=dev), km=torch.empty(Hkv, n[1], D, device=dev))

    if op == "select":
        return dict(case=case, qm=normal(case["H"], case["nq"], case["D"]), km=normal(case["Hkv"], case["nk"], case["D"]),
                    idx=torch.empty(case["H"], case["nq"], case["topk"], dtype=torch.int32, device=dev),
                    count=torch.empty(case["H"], case["nq"], dtype=torch.int32, device=dev))

    H, Hkv, Sq, Sk, D, ty = case["H"], case["Hkv"], case["Sq"], case["Sk"], case["D"], TYPES[case["type"]]
    nq, nk, cap = -(-Sq // QBLOCK), -(-Sk // case["block"]), case["cap"]
    count = torch.from_numpy(_counts(case)).to(dev)
    lists = torch.rand(H, nq, nk, generator=g, device=dev).topk(cap).indices      # distinct blocks
    lists = torch.where(torch.arange(cap, device=dev) < count[..., None], lists, nk).sort(-1).values
    idx = torch.where(lists < nk, lists, -1).to(torch.int32)
    # normalised queries and keys: logits of unit variance after the 1/sqrt(D) scale
    return dict(case=case, Q=normal(H, Sq, D).to(ty), K=normal(Hkv, Sk, D).to(ty), V=normal(Hkv, Sk, D).to(ty),
                idx=idx, count=count, O=torch.empty(H, Sq, D, dtype=ty, device=dev),
                L=torch.empty(H, Sq, device=dev), status=torch.zeros(4, dtype=torch.int32, device=dev))


# ----------------------------------------------------------------- the passes
def run(state):
    op = state["case"]["op"]
    return (_own if own else {"rope": _rope, "norm": _norm, "select": _select, "attend": _attend}[op])(state)


def _own(s):
    import partitioned_attention_state_b200 as dt

    c = s["case"]
    if c["op"] == "rope":
        dt.dt_rope_table(dt.rope_params(c["S"], s["axes"]), s["pos"], s["table"])
        return {"table": s["table"]}
    if c["op"] == "norm":
        x, H, Hkv = s["x"].transpose(0, 1), c["H"], c["Hkv"]                  # [heads][S][D] views of the projection
        q, k, v = x[:H], x[H:H + Hkv], x[H + Hkv:]
        qm, km = (s["qm"], s["km"]) if c["means"] else (None, None)
        p = dt.norm_rope_params(q, k, v, s["Q"], s["K"], s["V"], rot=c["rot"],
                                pairing=dt.DT_ROPE_HALVES if c["halves"] else dt.DT_ROPE_INTERLEAVED,
                                q_block=QBLOCK, k_block=c["block"])
        dt.dt_qk_norm_rope(p, q, k, v, s["wq"], s["wk"], s["table"], s["Q"], s["K"], s["V"], qm, km)
        return {n: s[n] for n in ("Q", "K", "V") + (("qm", "km") if c["means"] else ())}
    if c["op"] == "select":
        p = dt.select_params(c["H"], c["Hkv"], c["nq"], c["nk"], c["D"], c["topk"], c["first"], c["last"], c["margin"])
        dt.dt_block_select(p, s["qm"], s["km"], s["idx"], s["count"])
        return {"idx": s["idx"], "count": s["count"]}
    p = dt.sparse_params(s["Q"], s["K"], s["V"], s["O"], k_block=c["block"], cap=c["cap"])
    dt.dt_attn_block_sparse(p, s["Q"], s["K"], s["V"], s["idx"], s["count"], s["O"], s["L"], s["status"])
    return {"O": s["O"], "L": s["L"]}


def _rope(s):
    # angles of far positions lose their fraction in 32 bits: 64 throughout
    axes = torch.tensor(s["axes"], device=s["pos"].device)
    axis = torch.repeat_interleave(torch.arange(len(s["axes"]), device=s["pos"].device), axes // 2)
    i = torch.arange(len(axis), device=s["pos"].device) - (torch.cumsum(axes // 2, 0) - axes // 2)[axis]
    freq = torch.pow(10000.0, -2.0 * i.double() / axes[axis])
    angle = s["pos"][axis].T.double() * freq
    return {"table": torch.stack([angle.cos(), angle.sin()], -1).float()}


def _block_mean(x, block):
    n = x.shape[1]
    pad = torch.nn.functional.pad(x, (0, 0, 0, -n % block)).view(x.shape[0], -1, block, x.shape[2])
    rows = torch.clamp(n - block * torch.arange(pad.shape[1], device=x.device), max=block)
    return pad.sum(2) / rows[:, None]


def _norm_rotate(x, w, s, c):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    cos, sin, r = s["table"][..., 0], s["table"][..., 1], c["rot"]
    if c["halves"]:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1)


def _norm(s):
    c = s["case"]
    x, H, Hkv, out = s["x"].transpose(0, 1), c["H"], c["Hkv"], TYPES[c["out"]]
    q = _norm_rotate(x[:H].float(), s["wq"], s, c)
    k = _norm_rotate(x[H:H + Hkv].float(), s["wk"], s, c)
    res = {"Q": q.to(out), "K": k.to(out), "V": x[H + Hkv:].to(out).contiguous()}
    if c["means"]:
        res |= {"qm": _block_mean(q, QBLOCK), "km": _block_mean(k, c["block"])}
    return res


def _select(s):
    c = s["case"]
    nk, first, last = c["nk"], c["first"], c["last"]
    # scores next to the k-th decide a whole number: 64 bits
    km = s["km"].double().repeat_interleave(c["H"] // c["Hkv"], 0)
    score = s["qm"].double() @ km.transpose(1, 2) * (1.0 / math.sqrt(c["D"]))
    block = torch.arange(nk, device=score.device)
    forced = (block < first) | (block >= nk - last)
    order = torch.sort(torch.where(forced, math.inf, score), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, block.expand_as(order).contiguous())
    keep = rank < c["topk"]
    if c["margin"] < NO_MARGIN:
        keep &= forced | (score >= score.amax(-1, keepdim=True) - c["margin"])
    lists = torch.where(keep, block, nk).sort(-1).values[..., :c["topk"]]
    return {"idx": torch.where(lists < nk, lists, -1).to(torch.int32), "count": keep.sum(-1).to(torch.int32)}


def _attend(s):
    c = s["case"]
    H, Sq, Sk, D, block, dev = c["H"], c["Sq"], c["Sk"], c["D"], c["block"], s["Q"].device
    rows = min(QBLOCK, Sq)
    nq = -(-Sq // rows)
    q = torch.nn.functional.pad(s["Q"].float(), (0, 0, 0, nq * rows - Sq)).view(H, nq, rows, D)
    head = (torch.arange(H, device=dev) // (H // c["Hkv"]))[:, None, None]
    key = (s["idx"].long().clamp(min=0)[..., None] * block + torch.arange(block, device=dev)).flatten(-2)
    live = (torch.arange(c["cap"], device=dev) < s["count"][..., None]).repeat_interleave(block, -1) & (key < Sk)
    key = key.clamp(max=Sk - 1)
    p = torch.matmul(q, s["K"][head, key].float().transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    p.masked_fill_(~live[:, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, s["V"][head, key].float()) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + total.log())
    return {"O": o.flatten(1, 2)[:, :Sq].to(s["O"].dtype), "L": lse.flatten(1, 3)[:, :Sq].contiguous()}


# ----------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        pairs = sum(int(a) for a in case["axes"].split(",")) // 2
        # an angle (product), a cosine and a sine a pair
        return {"bytes": case["S"] * (8 * pairs + 4 * len(case["axes"].split(","))), "flops": 3 * case["S"] * pairs}
    if op == "norm":
        S, D, heads = case["S"], case["D"], case["H"] + case["Hkv"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        b = S * (heads + case["Hkv"]) * D * (size[case["type"]] + size[case["out"]]) + 4 * S * case["rot"] + 8 * D
        if case["means"]:
            b += 4 * D * (case["H"] * -(-S // QBLOCK) + case["Hkv"] * -(-S // case["block"]))
        # square, sum, two scalings; four products and two sums a pair
        return {"bytes": b, "flops": S * heads * (4 * D + 3 * case["rot"])}
    if op == "select":
        n = case["H"] * case["nq"]
        return {"bytes": 4 * case["D"] * (n + case["Hkv"] * case["nk"]) + 4 * n * (case["topk"] + 1),
                "flops": 2 * n * case["nk"] * case["D"]}
    Sq, Sk, D, block = case["Sq"], case["Sk"], case["D"], case["block"]
    count, nk = _counts(case), -(-Sk // block)
    rows = np.minimum(QBLOCK, Sq - QBLOCK * np.arange(count.shape[1]))
    keys = count * (Sk / nk)                                    # a list's keys, its blocks equally likely
    # expected share of the key rows that the lists of one key head name between them
    unread = np.prod((1 - count / nk).reshape(case["Hkv"], -1), axis=1)
    read = 2 * 2 * D * Sk * float((1 - unread).sum())
    return {"bytes": int(read + case["H"] * Sq * (4 * D + 4) + 4 * count.sum() + 4 * count.size),
            "flops": int(4 * D * (keys * rows).sum())}


# -------------------------------------------------------- the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "rope":
        cols = []
        for p, dim in zip(s["pos"].cpu().numpy().astype(np.float64), s["axes"]):
            cols.append(np.outer(p, 10000.0 ** (-np.arange(0, dim, 2) / dim)))
        angle = np.concatenate(cols, 1)
        return {"table": np.stack([np.cos(angle), np.sin(angle)], -1)}
    if op == "norm":
        H, Hkv, r = case["H"], case["Hkv"], case["rot"]
        turn = torch.view_as_complex(s["table"].to(f64).contiguous())
        res = {}
        for name, lo, n, w, m, block in (("Q", 0, H, "wq", "qm", QBLOCK), ("K", H, Hkv, "wk", "km", case["block"])):
            heads, means = [], []
            for h in range(lo, lo + n):                         # a head at a time: 64 bits are four times the input
                x = s["x"][:, h].to(f64)
                y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"] + 1e-6) * s[w].to(f64)
                pair = y[:, :r].reshape(-1, 2, r // 2).transpose(1, 2) if case["halves"] else y[:, :r].reshape(-1, r // 2, 2)
                z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
                y[:, :r] = (z.transpose(1, 2) if case["halves"] else z).reshape(-1, r)
                heads.append(y)
                means.append(torch.stack([b.mean(0) for b in y.split(block)]))
            res[name] = torch.stack(heads)
            res[m] = torch.stack(means)
        res["V"] = s["x"][:, H + Hkv:].transpose(0, 1).to(f64)
        return {n: res[n] for n in ("Q", "K", "V") + (("qm", "km") if case["means"] else ())}
    if op == "select":
        nk, topk, forced = case["nk"], case["topk"], set(range(case["first"])) | set(range(case["nk"] - case["last"], case["nk"]))
        q, k = s["qm"].cpu().numpy().astype(np.float64), s["km"].cpu().numpy().astype(np.float64)
        idx = np.full((case["H"], case["nq"], topk), -1, np.int32)
        count = np.zeros((case["H"], case["nq"]), np.int32)
        for h in range(case["H"]):
            score = q[h] @ k[h * case["Hkv"] // case["H"]].T / math.sqrt(case["D"])
            for i, row in enumerate(score):
                best = row.max()
                order = sorted(range(nk), key=lambda j: (j not in forced, -row[j], j))[:topk]
                kept = sorted(j for j in order if j in forced or row[j] >= best - case["margin"])
                idx[h, i, :len(kept)] = kept
                count[h, i] = len(kept)
        return {"idx": idx, "count": count}
    # every query against every key, the blocks that are not listed taken out
    H, Sq, Sk, D, block = case["H"], case["Sq"], case["Sk"], case["D"], case["block"]
    if H * Sq * Sk > 50e9:
        return None
    nk = -(-Sk // block)
    listed_ = torch.zeros(H, s["idx"].shape[1], nk + 1, dtype=torch.bool, device="cuda")
    listed_.scatter_(2, torch.where(s["idx"] < 0, nk, s["idx"]).long(), True)
    O = torch.zeros(H, Sq, D, dtype=f64, device="cuda")
    L = torch.full((H, Sq), -math.inf, dtype=f64, device="cuda")
    step = QBLOCK * max(1, (1 << 27) // (Sk * QBLOCK))
    for h in range(H):
        k, v = (s[n][h * case["Hkv"] // H].to(f64) for n in ("K", "V"))
        for a in range(0, Sq, step):
            b = min(Sq, a + step)
            seen = listed_[h, torch.arange(a, b, device="cuda") // QBLOCK, :nk].repeat_interleave(block, 1)[:, :Sk]
            z = torch.where(seen, s["Q"][h, a:b].to(f64) @ k.T / math.sqrt(D), -math.inf)
            L[h, a:b] = torch.logsumexp(z, 1)
            O[h, a:b] = torch.nan_to_num(torch.softmax(z, 1)) @ v      # a row with no keys gives 0
    return {"O": O, "L": L}
