"""The operators of the paged compressed key-value cache: what is measured, in plain torch and through the library.

Three operators around one cache of TurboQuant-MSE rows in pages:

  append   new tokens' keys and values are rotated, quantised, packed and written to their slots;
  decode   attention of one new token per sequence over the pages, with the weight each slot received added to `mass`;
  evict    the cache of each sequence and head is cut to a budget of slots by that accumulated weight.

Where `own` is false, run() computes them with elementary torch operations; where it is true it calls the library.
"""
import functools
import math

import numpy as np
import torch

own = False

D = 128          # head dimension of every configuration of this repository
KV_HEADS = 8     # KV heads of its grouped-query workload


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One user in the middle of a chat: a single sequence, short context; latency is all that counts.
        dict(name="decode_one_1021", op="decode", B=1, H=8, G=4, length=1021, ragged=False, page=16, kb=3, vb=3, dtype="bf16", mass=False),
        # A batch of conversations of all lengths (one of them just opened: no token yet), the weights kept for eviction.
        dict(name="decode_batch_mass_8191", op="decode", B=16, H=8, G=4, length=8191, ragged=True, page=64, kb=3, vb=3, dtype="bf16", mass=True),
        # One long document: the split over the length has to fill the machine from 8 heads.
        dict(name="decode_long_131072", op="decode", B=1, H=8, G=4, length=131072, ragged=False, page=128, kb=3, vb=3, dtype="bf16", mass=False),
        # A full server: 32 sequences of 32768 tokens, 64 query heads on 8 KV heads, 4-bit keys.
        dict(name="decode_server_32x32768", op="decode", B=32, H=8, G=8, length=32768, ragged=False, page=64, kb=4, vb=3, dtype="bf16", mass=False),
        # No grouping (one query head per KV head), fp32 queries and outputs, narrow keys and wide values.
        dict(name="decode_mha_f32_2049", op="decode", B=8, H=32, G=1, length=2049, ragged=True, page=32, kb=2, vb=4, dtype="f32", mass=False),
        # An odd group of heads (7 on each of 2), odd lengths, the smallest pages, with the weights.
        dict(name="decode_g7_mass_12345", op="decode", B=5, H=2, G=7, length=12345, ragged=True, page=16, kb=2, vb=2, dtype="bf16", mass=True),
        # The write of one decode step: one token of each of 64 sequences.
        dict(name="append_step_64", op="append", B=64, H=8, tokens=1, page=64, kb=3, vb=3, dtype="bf16"),
        # A prompt of one sequence.
        dict(name="append_prompt_8192", op="append", B=1, H=8, tokens=8192, page=64, kb=3, vb=3, dtype="bf16"),
        # Prompts of an odd length in fp32 at the widest codes.
        dict(name="append_f32_3x5001", op="append", B=3, H=8, tokens=5001, page=16, kb=4, vb=4, dtype="f32"),
        # One short conversation cut back to 512 slots.
        dict(name="evict_one_600_512", op="evict", B=1, H=8, length=600, budget=512, recent=32, page=16, kb=3, vb=3),
        # The steady state of a bounded cache: every 128 tokens, 16 sequences go back to 4096 slots.
        dict(name="evict_step_16x4224", op="evict", B=16, H=8, length=4224, budget=4096, recent=128, page=64, kb=3, vb=3),
        # The end of long prompts: a quarter of the tokens is kept.
        dict(name="evict_prompt_4x131072", op="evict", B=4, H=8, length=131072, budget=32768, recent=1024, page=128, kb=3, vb=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "append", "evict"))
    H = rng.choice((1, 2, 4, 8, 16))
    common = dict(op=op, H=H, page=rng.choice((16, 32, 64, 128, 256)), kb=rng.choice((2, 3, 4)), vb=rng.choice((2, 3, 4)))
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(common, B=B, tokens=_log(rng, 1, max(1, 8192 * 8 // (B * H))), dtype=rng.choice(("bf16", "f32")))
    B = _log(rng, 1, 64)
    longest = min(131072, 4194304 // (B * H))
    if op == "evict":
        length = _log(rng, 16, longest)
        budget = _log(rng, 8, length)
        return dict(common, B=B, length=length, budget=budget, recent=rng.randint(0, budget))
    return dict(common, B=B, G=rng.randint(1, 8), length=_log(rng, 1, longest), ragged=rng.random() < 0.6,
                dtype=rng.choice(("bf16", "bf16", "f32")), mass=rng.random() < 0.5)


def _lengths(case):
    """Tokens of each sequence. Ragged: spread evenly from none to the longest."""
    B, L = case["B"], case["length"]
    if not case.get("ragged") or B == 1:
        return [L] * B
    return [L * i // (B - 1) for i in range(B)]


def work(case):
    B, H, row = case["B"], case["H"], 16 * case["kb"] + 16 * case["vb"] + 4
    if case["op"] == "append":
        n = B * case["tokens"] * H
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (2 * D * e + row + 8) + 2 * H * D * D * 4 + 12 * B * case["tokens"], "flops": 4 * n * D * D}
    if case["op"] == "decode":
        e = 2 if case["dtype"] == "bf16" else 4
        T = sum(_lengths(case)) * H
        q = B * H * case["G"]
        return {"bytes": T * (row + (8 if case["mass"] else 0)) + 2 * q * D * e + 2 * H * D * D * 4,
                "flops": 4 * T * case["G"] * D + 4 * q * D * D}
    # evict: the expected number of moved rows, kept slots being spread over the sequence but for the recent ones
    L, keep, recent = case["length"], min(case["length"], case["budget"]), case["recent"]
    moved = min(recent, L - keep) + max(0, L - keep - recent) * max(0, keep - recent) / max(1, L - recent)
    return {"bytes": B * H * (8 * L + 8 * keep + 2 * row * moved), "flops": B * H * L}


# ---------------------------------------------------------------- inputs

@functools.lru_cache(maxsize=None)
def _codebook(bits):
    """Lloyd-Max centroids of one coordinate of a uniform unit vector in 128 dimensions."""
    x = np.linspace(-0.6, 0.6, 60001)
    w = (1 - x * x) ** ((D - 3) / 2)
    W, X = np.concatenate([[0.0], np.cumsum(w)]), np.concatenate([[0.0], np.cumsum(w * x)])
    c = np.linspace(-2, 2, 1 << bits) / math.sqrt(D)
    for _ in range(400):
        at = np.concatenate([[0], np.searchsorted(x, (c[1:] + c[:-1]) / 2), [len(x)]])
        c = (X[at[1:]] - X[at[:-1]]) / np.maximum(W[at[1:]] - W[at[:-1]], 1e-300)
    return c.astype(np.float32)


def _rotations(rs, H):
    return np.stack([np.linalg.qr(rs.standard_normal((D, D)))[0] for _ in range(H)]).astype(np.float32)


def _pack(codes, bits):
    """[..., 128] whole numbers -> [..., 16 * bits] bytes: code d in the stream's bits bits*d and up, low bits first."""
    t = (codes.to(torch.uint8).unsqueeze(-1) >> torch.arange(bits, dtype=torch.uint8, device=codes.device)) & 1
    t = t.reshape(*codes.shape[:-1], 16 * bits, 8) << torch.arange(8, dtype=torch.uint8, device=codes.device)
    return t.sum(-1, dtype=torch.uint8)


def _cells(y, cb):
    """The number of midpoints of the codebook strictly below y."""
    c = cb.double()
    mid = (c[1:] + c[:-1]) * 0.5
    n = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for m in mid:
        n += y > m
    return n


def _planes(gen, dev, N, H, page, bits, cb, lognorm):
    """Pages of quantised rows: a pool of unit vectors in rotated coordinates, drawn from for each row, with log-normal lengths."""
    y = torch.randn(1 << 14, D, generator=gen, device=dev, dtype=torch.float64)
    pool = _pack(_cells(y / y.norm(dim=1, keepdim=True), cb), bits)
    pick = torch.randint(0, 1 << 14, (N * H * page,), generator=gen, device=dev, dtype=torch.int32)
    plane = pool[pick].view(N, H, page, 16 * bits)
    norm = math.sqrt(D) * torch.exp(lognorm * torch.randn(N, H, page, generator=gen, device=dev))
    return plane, norm.to(torch.float16)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rs = np.random.default_rng(seed)
    B, H, page, kb, vb = case["B"], case["H"], case["page"], case["kb"], case["vb"]
    S = case["tokens"] if case["op"] == "append" else case["length"]
    lens = [S] * B if case["op"] != "decode" else _lengths(case)
    rs.shuffle(lens)
    M = -(-S // page)
    N = B * M + 3
    table = np.full((B, M), -1, dtype=np.int32)      # entries behind a sequence's last page are never used
    ids = rs.permutation(N)
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = ids[b * M:b * M - (-n // page)]
    kcb, vcb = (torch.from_numpy(_codebook(b)).to(dev) for b in (kb, vb))
    kp, kn = _planes(gen, dev, N, H, page, kb, kcb, 0.25)
    vp, vn = _planes(gen, dev, N, H, page, vb, vcb, 0.4)
    s = dict(op=case["op"], kp=kp, kn=kn, vp=vp, vn=vn, kcb=kcb, vcb=vcb, table=torch.from_numpy(table).to(dev),
             Pk=torch.from_numpy(_rotations(rs, H)).to(dev), Pv=torch.from_numpy(_rotations(rs, H)).to(dev))
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}.get(case.get("dtype"))
    if case["op"] == "decode":
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["Q"] = torch.randn(B, H * case["G"], D, generator=gen, device=dev).mul_(1.5).to(dtype)
        s["mass"] = torch.rand(B, H, S, generator=gen, device=dev) if case["mass"] else None
    elif case["op"] == "append":
        # channels of one scale but for a few large ones, as keys have them
        w = torch.ones(D, device=dev)
        w[[3, 17, 64, 101]] = 8.0
        n = B * S
        s["K"] = (torch.randn(n, H, D, generator=gen, device=dev) * w).to(dtype)
        s["V"] = torch.randn(n, H, D, generator=gen, device=dev).to(dtype)
        seq = torch.arange(B, device=dev).repeat_interleave(S)
        slot = torch.arange(S, device=dev).repeat(B)
        s["rows"] = torch.stack([seq, slot, slot + 7], dim=1).to(torch.int32)
        s["mass"] = torch.rand(B, H, S, generator=gen, device=dev)
        s["positions"] = torch.full((B, H, S), -1, dtype=torch.int32, device=dev)
    else:
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        # a few slots hold much of the weight; slots are not in the order of their tokens
        s["mass"] = torch.exp(2.0 * torch.randn(B, H, S, generator=gen, device=dev))
        old = torch.rand(B, H, S - min(S, case["recent"]), generator=gen, device=dev).argsort(-1).to(torch.int32)
        new = torch.arange(old.shape[-1], S, dtype=torch.int32, device=dev).expand(B, H, -1)
        s["positions"] = torch.cat([old, new], dim=-1).contiguous()
        s["seen"] = torch.full((B,), S, dtype=torch.int32, device=dev)
        s["budget"], s["recent"] = case["budget"], case["recent"]
        s["mass_out"] = torch.zeros(B, H, S, device=dev)
        s["positions_out"] = torch.full((B, H, S), -1, dtype=torch.int32, device=dev)
    if own:
        from compressed_kv_cache_gb300 import tq
        s["cache"] = tq.PagedCache(kp, kn, vp, vn, s["Pk"], kcb, s["Pv"], vcb)      # a layer's handle, made once
        if case["op"] == "decode":      # scratch that a server keeps from step to step
            s["workspace"] = torch.empty(tq.decode_paged_workspace_bytes(B, H, case["G"], S, case["mass"]), dtype=torch.uint8, device=dev)
        elif case["op"] == "evict":
            s["workspace"] = torch.empty(tq.evict_paged_workspace_bytes(B, H, S, case["budget"]), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"decode": _decode, "append": _append, "evict": _evict}[s["op"]](s)


def _values(plane, cb):
    """The centroids that the packed codes stand for, [..., 128] fp32."""
    bits = plane.shape[-1] // 16
    t = (plane.unsqueeze(-1) >> torch.arange(8, dtype=torch.uint8, device=plane.device)) & 1
    t = t.view(*plane.shape[:-1], D, bits) << torch.arange(bits, dtype=torch.uint8, device=plane.device)
    return cb[t.sum(-1, dtype=torch.uint8).int()]


def _gather(s, x):
    """[N, H, page, ...] -> [B, H, M * page, ...], the pages of each sequence in order (any page where there is none)."""
    t = x[s["table"].clamp(min=0).long()]
    t = t.transpose(1, 2)
    return t.reshape(t.shape[0], t.shape[1], t.shape[2] * t.shape[3], *t.shape[4:])


def _decode(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        out = tq.decode_paged(s["Q"], s["cache"], s["table"], s["lengths"], mass=s["mass"], workspace=s["workspace"])
        return {"out": out, "mass": s["mass"]}
    Q, H = s["Q"], s["Pk"].shape[0]
    B, G = Q.shape[0], Q.shape[1] // H
    a = torch.einsum("bhgj,hdj->bhgd", Q.float().view(B, H, G, D), s["Pk"])
    z = torch.matmul(a, _values(_gather(s, s["kp"]), s["kcb"]).transpose(-1, -2))
    z = z * _gather(s, s["kn"]).float().unsqueeze(2) / math.sqrt(D)
    there = (torch.arange(z.shape[-1], device=z.device) < s["lengths"].unsqueeze(1)).view(B, 1, 1, -1)
    z = z.masked_fill(~there, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    w = torch.where(there, p * _gather(s, s["vn"]).float().unsqueeze(2), torch.zeros_like(p))
    acc = torch.matmul(w, _values(_gather(s, s["vp"]), s["vcb"]))
    out = torch.einsum("bhgd,hdj->bhgj", acc, s["Pv"]).reshape(B, H * G, D).to(Q.dtype)
    if s["mass"] is not None:
        s["mass"] += p.sum(2)[..., :s["mass"].shape[-1]]
    return {"out": out, "mass": s["mass"]}


def _quantised(x, Pi, cb):
    """Packed codes and fp16 lengths of the rows x [n, H, 128], in 64 bits: a coordinate may lie next to a midpoint."""
    x = x.double()
    n = x.square().sum(-1, keepdim=True).sqrt()
    y = torch.einsum("nhj,hdj->nhd", torch.where(n > 0, x / n, torch.zeros_like(x)), Pi.double())
    return _pack(_cells(y, cb), int(math.log2(cb.numel()))), n.squeeze(-1).to(torch.float16)


def _append(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        tq.append_paged(s["K"], s["V"], s["rows"], s["cache"], s["table"], mass=s["mass"], positions=s["positions"])
    else:
        seq, slot, pos = s["rows"].long().unbind(1)
        page = s["kp"].shape[2]
        at = s["table"].long()[seq, slot // page], slice(None), slot % page
        s["kp"][at], s["kn"][at] = _quantised(s["K"], s["Pk"], s["kcb"])
        s["vp"][at], s["vn"][at] = _quantised(s["V"], s["Pv"], s["vcb"])
        s["mass"][seq, :, slot] = 0.0
        s["positions"][seq, :, slot] = pos.to(torch.int32).unsqueeze(1).expand(-1, s["positions"].shape[1])
    # the planes hold whole numbers (packed cell indices); a cell that differs is an error
    return {k: s[k] for k in ("kp", "kn", "vp", "vn", "mass", "positions")}


def _evict(s):
    if own:
        from compressed_kv_cache_gb300 import tq
        tq.evict_paged(s["cache"], s["table"], s["lengths"], s["seen"], s["mass"], s["positions"], s["budget"], s["recent"],
                       workspace=s["workspace"], out=(s["mass_out"], s["positions_out"]))
    else:
        mass, pos, page = s["mass"], s["positions"], s["kp"].shape[2]
        S = mass.shape[-1]
        slot = torch.arange(S, device=mass.device)
        length = s["lengths"].view(-1, 1, 1)
        keep = length.clamp(max=s["budget"])
        rank = (slot < length).int() + ((slot < length) & (pos >= s["seen"].view(-1, 1, 1) - s["recent"])).int()
        order = torch.sort(mass.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf), dim=-1, descending=True, stable=True).indices
        order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, descending=True, stable=True).indices)
        kept = torch.zeros(mass.shape, dtype=torch.bool, device=mass.device).scatter_(-1, order, slot.expand(mass.shape) < keep)
        # as many slots below `keep` are given up as kept ones lie behind it; both lists ascend, row by row
        b, h, to = ((slot < keep) & ~kept).nonzero(as_tuple=True)
        _, _, fro = ((slot >= keep) & kept).nonzero(as_tuple=True)
        table = s["table"].long()
        dst, src = (table[b, to // page], h, to % page), (table[b, fro // page], h, fro % page)
        for x in ("kp", "kn", "vp", "vn"):
            s[x][dst] = s[x][src]
        below = slot < keep
        for x, y in (("mass", "mass_out"), ("positions", "positions_out")):
            t = s[x].clone()
            t[b, h, to] = s[x][b, h, fro]
            s[y].copy_(torch.where(below, t, s[y]))
    return {k: s[k] for k in ("kp", "kn", "vp", "vn", "mass_out", "positions_out")}


# ---------------------------------------------------------------- in 64 bits

def _codes(rows, bits):
    """Codes of packed rows [n, 16 * bits], each taken from the 16 bits that it lies in."""
    first = torch.arange(D, device=rows.device) * bits
    wide = torch.cat([rows, torch.zeros_like(rows[:, :1])], dim=1).int()
    return ((wide[:, first // 8] | wide[:, first // 8 + 1] << 8) >> (first % 8).int()) & ((1 << bits) - 1)


def exact(case, seed):
    s = prepare(case, seed)
    page, H = case["page"], case["H"]
    if case["op"] == "append":
        kn, vn = s["kn"].double(), s["vn"].double()
        mass = s["mass"].double()
        mass.zero_()       # every slot is written
        for b in range(case["B"]):
            slot = torch.arange(case["tokens"], device=kn.device)
            pages = s["table"][b].long()[slot // page]
            of = slice(b * case["tokens"], (b + 1) * case["tokens"])
            for x, y in ((kn, s["K"]), (vn, s["V"])):
                x[pages, :, slot % page] = torch.linalg.vector_norm(y[of].double(), dim=-1)
        return {"kp": None, "kn": kn, "vp": None, "vn": vn, "mass": mass, "positions": None}
    if case["op"] == "decode":
        B, G = case["B"], case["G"]
        out = torch.zeros(B, H, G, D, dtype=torch.float64, device=s["Q"].device)
        mass = s["mass"].double() if s["mass"] is not None else None
        q = s["Q"].double().view(B, H, G, D)
        kc, vc = s["kcb"].double(), s["vcb"].double()
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // page)].long()
            for h in range(H):
                kp, vp = (s[x][pages, h].reshape(-1, s[x].shape[-1])[:n] for x in ("kp", "vp"))
                kn, vn = (s[x][pages, h].reshape(-1)[:n].double() for x in ("kn", "vn"))
                a = q[b, h] @ s["Pk"][h].double().T
                t = (kc[_codes(kp, case["kb"])] @ a.T) * (kn / D ** 0.5).unsqueeze(1)
                w = torch.softmax(t, dim=0)
                out[b, h] = (w.T @ (vc[_codes(vp, case["vb"])] * vn.unsqueeze(1))) @ s["Pv"][h].double()
                if mass is not None:
                    mass[b, h, :n] += w.sum(1)
        return {"out": out.view(B, H * G, D), "mass": mass}
    # evict: by one sort of each row in numpy
    B, S, budget = case["B"], case["length"], case["budget"]
    table = s["table"].cpu().numpy()
    mass, pos = s["mass"].cpu().numpy(), s["positions"].cpu().numpy()
    kn, vn = s["kn"].cpu().numpy().astype(np.float64), s["vn"].cpu().numpy().astype(np.float64)
    got = np.zeros((B, H, S))
    keep = min(S, budget)
    for b in range(B):
        for h in range(H):
            safe = pos[b, h] >= S - case["recent"]
            order = np.lexsort((np.arange(S), -mass[b, h].astype(np.float64), ~safe))
            chosen = np.sort(order[:keep])
            fro = chosen[chosen >= keep]
            to = np.setdiff1d(np.arange(keep), chosen)
            m = mass[b, h].astype(np.float64)
            m[to] = m[fro]
            got[b, h, :keep] = m[:keep]
            for x in (kn, vn):
                x[table[b, to // page], h, to % page] = x[table[b, fro // page], h, fro % page]
    return {"kp": None, "kn": kn, "vp": None, "vn": vn, "mass_out": got, "positions_out": None}
