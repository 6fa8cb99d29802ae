"""The operators of a decoder layer around the sparse FFN, as cases to measure.

Six kinds of call: the residual addition with its RMS norm (forward, with an output in 16, 32 or 8
bits, and backward), the paged key-value cache's write and its read-back, the attention of one new
token over that cache, and the matrix-vector product with 4-bit weights. Each case is one call of a
layer that is served (one to a few hundred tokens at once, contexts up to 131072 tokens) or trained
(batches of up to 16384 tokens) at the widths of this package's layers (d_model 2048 and 2560, heads
of 64 to 256) and at odd ones between.

`own = False` runs the plain forms: elementary torch operations in 32 bits, rounded once at the end.
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -60  # rows quieter than this are scaled as if this were their largest value
EPS = 1e-6


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a served layer: the latency of a call
        dict(name="norm_one_token", op="norm_fwd", N=1, d=2048, dtype="bf16", res="bf16", out="same", group=0),
        # a prompt or training batch, residual stream in 32 bits, the norm's output in 8 bits by 128 columns
        dict(name="norm_batch_8bit", op="norm_fwd", N=16384, d=2560, dtype="bf16", res="f32", out="e4m3", group=128),
        # backward of a small odd batch, gradients in 16 bits
        dict(name="norm_grad_small", op="norm_bwd", N=200, d=1000, dtype="bf16", res="bf16", grad="bf16", dh=False),
        # backward of a training batch behind the FFN's backward, whose dx is in 32 bits
        dict(name="norm_grad_batch", op="norm_bwd", N=16384, d=2560, dtype="bf16", res="f32", grad="f32", dh=True),
        # the new tokens of a decode batch go into the cache
        dict(name="append_decode", op="append", N=16, Hkv=4, hd=128, page=16, pages=2048, cache="e4m3", seqs=16),
        # a prompt's keys and values go into the cache, quantised
        dict(name="append_prompt", op="append", N=16001, Hkv=8, hd=128, page=64, pages=512, cache="e4m3", seqs=3),
        # a stored prefix is read back in 16 bits for a later prompt that continues it
        dict(name="gather_prefix", op="gather", N=30011, Hkv=8, hd=128, page=64, pages=1024, cache="e4m3", seqs=5),
        # a batch of short requests, lengths 0 to 200, small pages
        dict(name="attn_short_batch", op="attn", B=16, Hkv=4, G=4, hd=64, page=16, max_len=200, cache="bf16", window=0,
             ragged=True),
        # one request with a long context
        dict(name="attn_one_long", op="attn", B=1, Hkv=4, G=5, hd=128, page=64, max_len=131072, cache="bf16", window=0,
             ragged=False),
        # a busy server: ragged lengths, a cache in 8 bits
        dict(name="attn_busy_8bit", op="attn", B=64, Hkv=4, G=4, hd=128, page=64, max_len=16384, cache="e4m3", window=0,
             ragged=True),
        # the output projection of one token
        dict(name="w4_one_token", op="w4", N=1, k=2048, n=2048, group=128),
        # a wide projection for a decode batch, fine groups
        dict(name="w4_batch_wide", op="w4", N=16, k=2560, n=13824, group=32),
    ]


LARGEST = 536_870_912  # cache values of one kind that the largest attention case may hold (64 x 16384 x 4 x 128)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "append", "gather", "attn", "attn", "w4"])
    if op in ("norm_fwd", "norm_bwd"):
        d = 8 * _log_int(rng, 8, 1024)
        N = _log_int(rng, 1, min(65536, 16384 * 2560 // d))
        dtype, res = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "none")])
        if op == "norm_fwd":
            out = rng.choice(["same", "e4m3"])
            return dict(op=op, N=N, d=d, dtype=dtype, res=res, out=out, group=rng.choice([0, 128]) if out == "e4m3" else 0)
        res = "bf16" if res == "none" else res
        return dict(op=op, N=N, d=d, dtype=dtype, res=res, grad=rng.choice(["bf16", "f32"]), dh=rng.random() < 0.5)
    if op in ("append", "gather"):
        hd, Hkv = rng.choice([64, 96, 128, 256]), rng.randint(1, 20)
        page = rng.choice([1, 8, 16, 32, 64, 128])
        N = _log_int(rng, 1, 16384 * 1024 // (Hkv * hd))
        seqs = rng.randint(1, min(N, 32))
        pages = N // page + seqs + rng.randint(1, 64)
        return dict(op=op, N=N, Hkv=Hkv, hd=hd, page=page, pages=pages, cache=rng.choice(["bf16", "e4m3"]), seqs=seqs)
    if op == "attn":
        hd, Hkv, G = rng.choice([64, 96, 128, 256]), rng.choice([1, 2, 3, 4, 5, 8, 16, 20]), rng.choice([1, 2, 3, 4, 5, 7, 8, 10, 16, 20])
        B = _log_int(rng, 1, 256)
        # at most half of the largest case's values, for the 16-bit cache or many heads to a key less: a drawn case
        # costs no more than that one
        cache = rng.choice(["bf16", "e4m3"])
        most = LARGEST // (4 if cache == "bf16" else 2) // max(1, G // 4) // (B * Hkv * hd)
        max_len = _log_int(rng, 1, max(1, min(131072, most)))
        window = rng.choice([0, 0, _log_int(rng, 1, max_len)])
        return dict(op=op, B=B, Hkv=Hkv, G=G, hd=hd, page=rng.choice([8, 16, 32, 64, 128]), max_len=max_len, cache=cache,
                    window=window, ragged=rng.random() < 0.7)
    k = 32 * _log_int(rng, 2, 256)
    group = rng.choice([g for g in (32, 64, 128) if k % g == 0])
    return dict(op="w4", N=rng.randint(1, 16), k=k, n=_log_int(rng, 16, 16384), group=group)


# ------------------------------------------------------------------------------------------ inputs

def _lens(case):
    """The batch's context lengths: by the case alone. Ragged ones are spread over 0..max_len, the first of them
    max_len, the second 0, the third 1."""
    B, top = case["B"], case["max_len"]
    if not case["ragged"]:
        return [top] * B
    r = random.Random(1000 * B + top)
    lens = [r.randint(0, top) for _ in range(B)]
    for i, v in enumerate((top, 0, min(1, top))[:B]):
        lens[i] = v
    return lens


def _visible(case):
    w = case["window"]
    return [min(n, w) if w else n for n in _lens(case)]


def _seq_slots(N, seqs, page, pages, seed):
    """Slots of N tokens that belong to `seqs` sequences one after another, in pages drawn at random; the last token of
    each fifth sequence is a padding token without a slot."""
    r = np.random.RandomState(seed % (2 ** 31))
    perm = r.permutation(pages)
    slots, used = [], 0
    for i in range(seqs):
        n = N // seqs + (1 if i < N % seqs else 0)
        need = -(-n // page)
        pg = perm[used:used + need]
        used += need
        t = np.arange(n)
        s = pg[t // page] * page + t % page
        if n > 1 and i % 5 == 4:
            s[-1] = -1
        slots.append(s)
    return np.concatenate(slots).astype(np.int32)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32)


def _keys(g, *shape):
    """Keys or values as layers have them: normal, some channels ten times as large."""
    x = _normal(g, *shape)
    loud = 1 + 9 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.05).to(F32)
    return x * loud


def _cache(g, case, pages):
    """A cache filled with the keys and values of earlier tokens: bf16, or e4m3 codes with a scale a token and head."""
    shape = (pages, case["Hkv"], case["page"], case["hd"])
    out = {}
    for name in ("k", "v"):
        t = _keys(g, *shape)
        if case["cache"] == "bf16":
            out[name], out[name + "_scale"] = t.to(BF16), None
        else:
            a = t.abs().amax(-1).clamp_min(AMAX_MIN)
            out[name] = (t * (E4M3_MAX / a)[..., None]).to(E4M3)
            out[name + "_scale"] = a / E4M3_MAX
    return out


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": case}
    if op in ("norm_fwd", "norm_bwd"):
        N, d = case["N"], case["d"]
        dt, rt = DTYPES[case["dtype"]], DTYPES.get(case["res"])
        s["w"] = (1 + 0.2 * _normal(g, d)).to(dt)
        if op == "norm_fwd":
            s["x"] = _normal(g, N, d).to(dt)
            s["res"] = None if rt is None else (3 * _normal(g, N, d)).to(rt)
            ng = -(-d // case["group"]) if case["group"] else 1
            s["h"] = None if rt is None else torch.empty((N, d), dtype=rt, device="cuda")
            s["y"] = torch.empty((N, d), dtype=dt if case["out"] == "same" else E4M3, device="cuda")
            s["scale"] = torch.empty((N, ng), dtype=F32, device="cuda") if case["out"] == "e4m3" else None
        else:
            gt = DTYPES[case["grad"]]
            s["h"] = (3 * _normal(g, N, d)).to(rt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
            s["dy"] = _normal(g, N, d).to(gt)
            s["dh"] = _normal(g, N, d).to(gt) if case["dh"] else None
            s["dx"] = torch.empty((N, d), dtype=gt, device="cuda")
            s["dw"] = torch.empty((d,), dtype=F32, device="cuda")
    elif op in ("append", "gather"):
        s.update(_cache(g, case, case["pages"]))
        N, H, hd = case["N"], case["Hkv"], case["hd"]
        s["slots"] = torch.from_numpy(_seq_slots(N, case["seqs"], case["page"], case["pages"], int(seed))).cuda()
        if op == "append":
            # keys and values as the fused projection leaves them: slices of one row a token, behind as many queries
            qkv = _keys(g, N, 3 * H, hd).to(BF16)
            s["k_new"], s["v_new"] = qkv[:, H:2 * H], qkv[:, 2 * H:]
        else:
            s["k_out"], s["v_out"] = (torch.empty((N, H, hd), dtype=BF16, device="cuda") for _ in range(2))
    elif op == "attn":
        B, page = case["B"], case["page"]
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        s.update(_cache(g, case, pages))
        perm = np.random.RandomState(int(seed) % (2 ** 31)).permutation(pages)
        table = np.zeros((B, max(1, max(need))), dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        s["table"] = torch.from_numpy(table).cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal(g, B, case["Hkv"] * case["G"], case["hd"]).to(BF16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=F32, device="cuda")
    else:
        N, k, n, group = case["N"], case["k"], case["n"], case["group"]
        # the packed weights: tiles of 16 rows by 128 columns, each lane's 8 words next to each other (see _w4_codes)
        nt, kt = -(-n // 16), -(-k // 128)
        codes = torch.randint(0, 16, (nt * 16, kt * 128), generator=g, device="cuda", dtype=torch.int32)
        codes[n:] = 8
        codes[:, k:] = 8
        t = codes.view(nt, 2, 8, kt, 4, 4, 4, 2)  # tile, half, row, tile, j, c, pair, member
        t = t.permute(0, 3, 2, 5, 1, 4, 6, 7).contiguous()  # tile, tile, row, c, half, j, pair, member
        shift = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device="cuda", dtype=torch.int64)
        words = (t.to(torch.int64) << shift).sum((-1, -2))
        s["words"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)  # [nt, kt, 8, 4, 2, 4]
        sc = (0.5 + torch.rand((nt * 16, kt * 128 // group), generator=g, device="cuda")) / (4 * math.sqrt(k))
        sc[n:] = 0
        sc[:, k // group:] = 0
        s["scales"] = sc.view(nt, 2, 8, kt, 128 // group).permute(0, 3, 2, 1, 4).to(BF16).contiguous()
        s["x"] = _normal(g, N, k).to(BF16)
        s["y"] = torch.empty((N, n), dtype=BF16, device="cuda")
    if own:  # the handles that a program keeps beside its tensors
        from activation_sparse_ffn_gate_gb300 import binding
        s["lib"] = binding
        if "k_scale" in s:
            s["cache"] = binding.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "w4":
            s["weights"] = binding.W4Weights(s["words"], s["scales"], case["n"], case["k"], case["group"])
        if op == "norm_fwd" and case["out"] == "e4m3":
            s["y8"] = binding.Rows8(s["y"], s["scale"], case["group"])
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _to8(t, a):
    """t rounded to e4m3 under the largest absolute value a (with t's axes), and the scale."""
    a = a.clamp_min(AMAX_MIN)
    return (t * (E4M3_MAX / a)).to(E4M3), a / E4M3_MAX


def _norm_fwd(s):
    c = s["case"]
    h = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
    out = {} if s["res"] is None else {"h": h.to(s["res"].dtype)}
    if c["out"] == "same":
        return {**out, "y": y.to(s["x"].dtype)}
    N, d = y.shape
    group = c["group"] or d
    ng = -(-d // group)
    p = torch.nn.functional.pad(y, (0, ng * group - d)).view(N, ng, group)
    q, scale = _to8(p, p.abs().amax(-1, keepdim=True))
    return {**out, "y": q.view(N, ng * group)[:, :d], "scale": scale[..., 0]}


def _norm_bwd(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xh, gw = h * rstd, dy * s["w"].float()
    dx = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * xh).sum(0)}


def _append(s):
    c = s["case"]
    page = c["page"]
    at = s["slots"].long()
    keep = at >= 0
    pg, off = at[keep] // page, at[keep] % page
    for name in ("k", "v"):
        t = s[name + "_new"][keep]
        if c["cache"] == "bf16":
            s[name][pg, :, off] = t
        else:
            q, scale = _to8(t.float(), t.float().abs().amax(-1, keepdim=True))
            s[name].view(torch.uint8)[pg, :, off] = q.view(torch.uint8)
            s[name + "_scale"][pg, :, off] = scale[..., 0]
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}


def _rows(s, name, pg, off):
    """Rows of the cache at pages pg and offsets off, in 32 bits."""
    if s[name + "_scale"] is None:
        return s[name][pg, :, off].float()
    return s[name].view(torch.uint8)[pg, :, off].view(E4M3).float() * s[name + "_scale"][pg, :, off][..., None]


def _gather(s):
    at = s["slots"].long()
    keep = (at >= 0)[:, None, None]
    at = at.clamp_min(0)
    pg, off = at // s["case"]["page"], at % s["case"]["page"]
    return {n + "_out": torch.where(keep, _rows(s, n, pg, off), 0.0).to(BF16) for n in ("k", "v")}


def _attn(s):
    c = s["case"]
    B, H, G, hd = c["B"], c["Hkv"], c["G"], c["hd"]
    L = s["table"].shape[1] * c["page"]
    pos = torch.arange(L, device="cuda")[None, :]
    lens = s["lens"].long()[:, None]
    seen = pos < lens
    if c["window"]:
        seen = seen & (pos >= lens - c["window"])

    def whole(name):  # [B, H, L, hd]
        if s[name + "_scale"] is None:
            t = s[name][s["table"].long()].float()
        else:
            t = s[name].view(torch.uint8)[s["table"].long()].view(E4M3).float()
            t *= s[name + "_scale"][s["table"].long()][..., None]
        return t.permute(0, 2, 1, 3, 4).reshape(B, H, L, hd)

    sc = torch.matmul(s["q"].float().view(B, H, G, hd), whole("k").transpose(-1, -2)) / math.sqrt(hd)
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - top.clamp_min(-3e38))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, whole("v")) / total.clamp_min(1e-30)
    lse = (top + total.log())[..., 0]
    return {"out": o.to(BF16).view(B, H * G, hd), "lse": lse.view(B, H * G)}


def _w4_codes(s):
    """Codes 0..15 and scales as [rows, columns] from the packed words: a tile's 16 rows are two halves of 8, its 128
    columns 4 groups j of 4 lanes c of 8, and a word holds its column 2i in bits 4i.. and its column 2i+1 in bits 16+4i.."""
    nt, kt = s["words"].shape[:2]
    shift = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device="cuda", dtype=torch.int32)
    t = (s["words"][..., None, None] >> shift) & 15  # tile, tile, row, c, half, j, pair, member
    codes = t.permute(0, 4, 2, 1, 5, 3, 6, 7).reshape(nt * 16, kt * 128)
    scales = s["scales"].permute(0, 3, 2, 1, 4).reshape(nt * 16, -1)
    return codes, scales


def _w4(s):
    c = s["case"]
    codes, scales = _w4_codes(s)
    W = (codes - 8).float() * scales.float().repeat_interleave(c["group"], dim=1)
    return {"y": torch.matmul(s["x"].float(), W[:c["n"], :c["k"]].t()).to(BF16)}


# ------------------------------------------------------------------------------------------ the calls

def run(s):
    op, c = s["op"], s["case"]
    if not own:
        return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "append": _append, "gather": _gather, "attn": _attn,
                "w4": _w4}[op](s)
    lib = s["lib"]
    if op == "norm_fwd":
        if c["out"] == "same":
            y, h, _ = lib.twell_add_rmsnorm_fwd(s["x"], s["w"], s["res"], EPS, y=s["y"], h=s["h"])
            return {"y": y} if h is None else {"h": h, "y": y}
        y8, h, _ = lib.twell_add_rmsnorm_fwd_q8(s["x"], s["w"], s["res"], EPS, out=s["y8"], h=s["h"])
        out = {"y": y8.values, "scale": y8.scale}
        return out if h is None else {"h": h, **out}
    if op == "norm_bwd":
        dx, dw = lib.twell_add_rmsnorm_bwd(s["dy"], s["h"], s["w"], s["rstd"], s["dh"], dx=s["dx"], dw=s["dw"])
        return {"dx": dx, "dw": dw}
    if op == "append":
        lib.twell_kv_append(s["cache"], s["k_new"], s["v_new"], s["slots"])
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}
    if op == "gather":
        k, v = lib.twell_kv_gather(s["cache"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
        return {"k_out": k, "v_out": v}
    if op == "attn":
        out, lse = lib.twell_paged_attn_decode(s["q"], s["cache"], s["table"], s["lens"], window=c["window"],
                                               out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    return {"y": lib.twell_w4_matvec(s["x"], s["weights"], y=s["y"])}


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "e4m3": 1, "none": 0}
    if op == "norm_fwd":
        N, d = case["N"], case["d"]
        b, r = size[case["dtype"]], size[case["res"]]
        o = b if case["out"] == "same" else 1
        ng = (-(-d // case["group"]) if case["group"] else 1) if case["out"] == "e4m3" else 0
        return {"bytes": N * d * (b + 2 * r + o) + 4 * N * ng + d * b, "flops": 6 * N * d}
    if op == "norm_bwd":
        N, d = case["N"], case["d"]
        b = size[case["grad"]]
        return {"bytes": N * d * (b * (3 if case["dh"] else 2) + size[case["res"]]) + 4 * N + d * (4 + size[case["dtype"]]),
                "flops": 12 * N * d}
    if op in ("append", "gather"):
        N, row = case["N"] * case["Hkv"], case["hd"]
        e = 2 * row if case["cache"] == "bf16" else row + 4
        return {"bytes": 2 * N * (2 * row + e) + 4 * case["N"], "flops": 4 * N * row}
    if op == "attn":
        H, G, hd = case["Hkv"], case["G"], case["hd"]
        seen = sum(_visible(case))
        e = 2 * hd if case["cache"] == "bf16" else hd + 4
        pages = sum(-(-n // case["page"]) for n in _visible(case))
        return {"bytes": 2 * seen * H * e + 4 * pages + case["B"] * (4 + H * G * (4 * hd + 4)), "flops": 4 * seen * H * G * hd}
    N, k, n = case["N"], case["k"], case["n"]
    return {"bytes": n * k // 2 + 2 * n * (k // case["group"]) + 2 * N * (n + k), "flops": 2 * N * n * k}


# ------------------------------------------------------------------------------------------ 64 bits

def _near8(v):
    """The e4m3 values nearest to v (64 bits, |v| at most a hair over 448), ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _row64(s, name, slot, page):
    """[n, Hkv, hd] in 64 bits: cache rows by slot."""
    pg, off = torch.div(slot, page, rounding_mode="floor"), slot % page
    if s[name].dtype == BF16:
        return s[name][pg, :, off].double()
    return s[name].view(torch.uint8)[pg, :, off].view(E4M3).double() * s[name + "_scale"][pg, :, off].double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        h = s["x"].double()
        if s["res"] is not None:
            h = h + s["res"].double()
        rms = (h.pow(2).sum(1) / case["d"] + EPS).sqrt()
        y = h / rms[:, None] * s["w"].double()
        out = {} if s["res"] is None else {"h": h}
        if case["out"] == "same":
            return {**out, "y": y}
        width = case["group"] or case["d"]
        ys, scales = [], []
        for part in y.split(width, dim=1):
            a = part.abs().max(1, keepdim=True).values.clamp_min(AMAX_MIN)
            ys.append(_near8(part * (E4M3_MAX / a)))
            scales.append(a / E4M3_MAX)
        return {**out, "y": torch.cat(ys, 1), "scale": torch.cat(scales, 1)}
    if op == "norm_bwd":
        # y_i = h_i w_i / r with r^2 = mean(h^2) + eps; s["rstd"] is that 1/r
        inv = s["rstd"].double()[:, None]
        h, t = s["h"].double(), s["dy"].double() * s["w"].double()
        dx = t * inv - h * inv.pow(3) * (t * h).sum(1, keepdim=True) / case["d"]
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("nd,nd,nx->d", s["dy"].double(), h, inv)}
    if op == "append":
        out = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}
        live = (s["slots"] >= 0).nonzero()[:, 0]
        slot = s["slots"][live].long()
        pg, off = torch.div(slot, case["page"], rounding_mode="floor"), slot % case["page"]
        for n in ("k", "v"):
            t = s[n + "_new"][live].double()
            if case["cache"] == "e4m3":
                a = t.abs().max(2).values.clamp_min(AMAX_MIN)
                out[n + "_scale"][pg, :, off] = a / E4M3_MAX
                t = _near8(t * (E4M3_MAX / a)[..., None])
            out[n][pg, :, off] = t
        return out
    if op == "gather":
        out = {}
        live = (s["slots"] >= 0).nonzero()[:, 0]
        for n in ("k", "v"):
            o = torch.zeros((case["N"], case["Hkv"], case["hd"]), dtype=torch.float64, device="cuda")
            o[live] = _row64(s, n, s["slots"][live].long(), case["page"])
            out[n + "_out"] = o
        return out
    if op == "attn":
        B, H, G, hd, page = case["B"], case["Hkv"], case["G"], case["hd"], case["page"]
        out = torch.zeros((B, H, G, hd), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, G), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            pos = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            slot = s["table"][b, pos // page].long() * page + pos % page
            q = s["q"][b].double().view(H, G, hd)
            z = torch.einsum("hgd,nhd->hgn", q, _row64(s, "k", slot, page)) * hd ** -0.5
            lse[b] = torch.logsumexp(z, -1)
            out[b] = torch.einsum("hgn,nhd->hgd", torch.exp(z - lse[b][..., None]), _row64(s, "v", slot, page))
        return {"out": out.view(B, H * G, hd), "lse": lse.view(B, H * G)}
    # one row of 16 x 128 tiles at a time, by the words' bits
    nt, kt = s["words"].shape[:2]
    x = torch.zeros((case["N"], kt * 128), dtype=torch.float64, device="cuda")
    x[:, :case["k"]] = s["x"].double()
    x = x.view(case["N"], kt, 4, 4, 8)  # token, tile, j, c, column
    bits = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda", dtype=torch.int32)
    rows = torch.zeros((nt, 2, 8, case["N"]), dtype=torch.float64, device="cuda")
    per = 4 // (128 // case["group"])
    for i in range(nt):
        code = ((s["words"][i][..., None] >> bits) & 15).double() - 8  # tile, row, c, half, j, column
        part = torch.einsum("trchjm,ntjcm->thrjn", code, x)  # tile, half, row, j, token
        sc = s["scales"][i].double().repeat_interleave(per, dim=3)  # tile, row, half, j
        rows[i] = torch.einsum("thrjn,trhj->hrn", part, sc)
    return {"y": rows.view(nt * 16, case["N"])[:case["n"]].t().contiguous()}
