"""What a served or trained step needs beside a decoder layer's own calls, as cases to measure.

Three kinds of call: the rotation of queries and keys by their positions (forward for serving, backward for
training; both pair layouts, the whole head or part of it, frequencies scaled for long contexts), the plan of a step
on the device (pages of new tokens taken from a pool of free ones, those of ended requests put back, and the slot,
position and label of each of the step's tokens), and the low-rank adapters of many requests added to a
shared projection's output. Sizes are those of this package's layers (d_model 2048 and 2560, heads of 64 to 256), one token to
long prompts, and odd ones between.

`own = False` runs the plain forms: elementary torch operations in 32 bits (the angles in 64), rounded once at the end.
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
DTYPES = {"bf16": BF16, "f32": F32}


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a served layer: the latency of a call; q and k are views of the fused projection
        dict(name="rope_one_token", op="rope", way="fwd", form="rows", B=1, S=1, Hq=16, Hk=8, hd=128, rot=128, pairs="half",
             dtype="bf16", scaling="none", far=4000),
        # a decode batch far into long contexts: half of each head turns, neighbours are pairs
        dict(name="rope_decode_far", op="rope", way="fwd", form="rows", B=1, S=250, Hq=20, Hk=4, hd=128, rot=64,
             pairs="neighbours", dtype="bf16", scaling="bands", far=1_000_000),
        # the prompts of a few requests
        dict(name="rope_prompt", op="rope", way="fwd", form="rows", B=1, S=16001, Hq=16, Hk=8, hd=128, rot=128, pairs="half",
             dtype="bf16", scaling="ramp", far=100_000),
        # backward of a training batch, head-first gradients in 32 bits, three quarters of each head turn
        dict(name="rope_grad_batch", op="rope", way="bwd", form="heads", B=4, S=4096, Hq=20, Hk=4, hd=128, rot=96, pairs="half",
             dtype="f32", scaling="none", far=4096),
        # a decode step of a small batch, small pages
        dict(name="plan_decode", op="plan", B=16, page=16, past=4000, new="one", pad=0),
        # a busy server's step: most requests decode, some bring a piece of their prompt, some have ended
        dict(name="plan_busy", op="plan", B=500, page=64, past=16384, new="mixed", pad=77),
        # long prompts arrive at once
        dict(name="plan_prompts", op="plan", B=37, page=64, past=0, new="prompts", pad=0),
        # one token of one request
        dict(name="lora_one_token", op="lora", N=1, k=2048, n=2048, R=16, L=8, form="decode", ranks="full", wide=False),
        # a decode batch, nearly every request with an adapter of its own, of other ranks
        dict(name="lora_decode_many", op="lora", N=64, k=2048, n=4096, R=64, L=64, form="decode", ranks="ragged", wide=False),
        # a larger decode batch that shares a few adapters; the output is a slice of a fused projection's
        dict(name="lora_decode_shared", op="lora", N=200, k=2560, n=2560, R=32, L=4, form="decode", ranks="full", wide=True),
        # pieces of prompts beside a decode batch
        dict(name="lora_mixed", op="lora", N=3001, k=2560, n=2568, R=24, L=40, form="mixed", ranks="ragged", wide=False),
        # prompts of a few requests
        dict(name="lora_prompts", op="lora", N=16384, k=2048, n=4096, R=16, L=8, form="prompts", ranks="full", wide=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


ROPE_VALUES = 4 * 4096 * 24 * 128  # of the largest rotation
PLAN_TOKENS = 2_000_000
LORA_VALUES = 16384 * (2048 + 2 * 4096)  # of x and y, read and written


def draw(rng):
    op = rng.choice(["rope", "rope", "plan", "lora", "lora"])
    if op == "rope":
        hd = rng.choice([32, 64, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4, 5, 7, 8])
        N = _log_int(rng, 1, min(32768, ROPE_VALUES // ((Hq + Hk) * hd)))
        form = rng.choice(["rows", "heads"])
        B = 1 if form == "rows" else rng.randint(1, min(N, 8))
        rot = rng.choice([hd, hd, hd // 2, hd // 4, 2 * rng.randint(1, hd // 2)])
        return dict(op=op, way=rng.choice(["fwd", "bwd"]), form=form, B=B, S=N // B, Hq=Hq, Hk=Hk, hd=hd, rot=rot,
                    pairs=rng.choice(["half", "neighbours"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    scaling=rng.choice(["none", "linear", "base", "bands", "ramp"]), far=_log_int(rng, 100, 2_000_000))
    if op == "plan":
        new = rng.choice(["one", "mixed", "prompts"])
        B = _log_int(rng, 1, {"one": 4096, "mixed": 2048, "prompts": 64}[new])
        return dict(op=op, B=B, page=rng.choice([1, 8, 16, 32, 64, 128, 256]) if new == "one" else rng.choice([16, 32, 64, 128]),
                    past=_log_int(rng, 1, min(131072, max(1, PLAN_TOKENS // B))), new=new, pad=rng.choice([0, rng.randint(1, 300)]))
    form = rng.choice(["decode", "decode", "mixed", "prompts"])
    k, n = 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 8, 1024)
    R = 8 * rng.choice([1, 2, 2, 3, 4, 4, 8, 8, 16])
    L = _log_int(rng, 1, 64)
    N = _log_int(rng, 1, 500) if form == "decode" else _log_int(rng, 64, min(16384, LORA_VALUES // (k + 2 * n), 2 ** 24 // (L * R)))
    return dict(op=op, N=N, k=k, n=n, R=R, L=L, form=form, ranks=rng.choice(["full", "ragged"]), wide=rng.random() < 0.4)


# ------------------------------------------------------------------------------------------ what a case stands for

BASE, FACTOR, ORIGINAL = 10000.0, 8.0, 8192  # of the rotations; the scaled ones serve eight times their trained length


def _frequencies(case):
    """Radians a position for each pair, in 64 bits, and the factor on the turned values."""
    rot, how = case["rot"], case["scaling"]
    i = np.arange(rot // 2, dtype=np.float64)
    base = BASE
    if how == "base" and rot > 2:
        base = BASE * FACTOR ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if how == "linear":
        return f / FACTOR, 1.0
    if how == "bands":  # waves shorter than a quarter of the trained length stay, those longer than it are stretched
        share = np.clip((ORIGINAL * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f * share + f / FACTOR * (1 - share), 1.0
    if how == "ramp":  # by the number of turns within the trained length: 32 and more stay, one and fewer are stretched

        def pair(turns):
            return rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _step(case):
    """The requests' tokens so far and new ones (-1: the request has ended), by the case alone."""
    B, top, r = case["B"], case["past"], random.Random(977 * case["B"] + case["past"])
    past = [r.randint(0, top) for _ in range(B)]
    new = [1] * B
    if case["new"] == "prompts":
        past = [0 if r.random() < 0.8 else p for p in past]
        most = min(131072, PLAN_TOKENS // B)
        new = [r.randint(1, most) for _ in range(B)]
        new[0] = most
    elif case["new"] == "mixed":
        for b in range(B):
            u = r.random()
            if u < 0.06:
                new[b] = r.randint(2, 900)
            elif u < 0.1:
                new[b] = -1
            elif u < 0.12:
                new[b] = 0
            if u < 0.03:
                past[b] = 0
    return past, new


def _ids(case):
    """Each token's adapter (-1: none), by the case alone."""
    N, L, r = case["N"], case["L"], random.Random(31 * case["N"] + case["L"])

    def one():
        return -1 if r.random() < 0.08 else r.randrange(L)
    if case["form"] == "decode":
        ids = [one() for _ in range(N)]
        ids[0] = L - 1
        return ids
    tail = min(N // 4, 150) if case["form"] == "mixed" else 0  # decode tokens behind the prompts
    pieces, ids = max(2, min(12, N // 200)), []
    for i in range(pieces):
        a = L - 1 if i == 0 else one()
        upto = (N - tail) * (i + 1) // pieces
        ids += [a] * (upto - len(ids))
    return ids + [one() for _ in range(tail)]


def _ranks(case):
    L, R, r = case["L"], case["R"], random.Random(case["L"] + 1000 * case["R"])
    if case["ranks"] == "full":
        return [R] * L
    return [min(R, r.choice([4, 8, 16, 32, 64, R, R])) for _ in range(L)]


# ------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    op = case["op"]
    rs = np.random.RandomState(int(seed) % (2 ** 31))
    s = {"op": op, "case": case}
    if op == "rope":
        B, S, Hq, Hk, hd, t = case["B"], case["S"], case["Hq"], case["Hk"], case["hd"], DTYPES[case["dtype"]]
        freq, s["factor"] = _frequencies(case)
        s["freq"] = torch.from_numpy(freq).cuda()
        if case["form"] == "rows":
            # rows of the fused projection: queries, keys, values; a decode batch or the pieces of a few prompts
            rows = _normal(g, S, Hq + 2 * Hk, hd).to(t)
            s["q"], s["k"] = rows[:, :Hq], rows[:, Hq:Hq + Hk]
            if S <= 512:
                pos = rs.randint(0, case["far"], size=S)
            else:
                starts = rs.randint(0, max(1, case["far"]), size=5)
                pos = np.concatenate([p + np.arange(len(c)) for p, c in zip(starts, np.array_split(np.arange(S), 5))])
        else:
            s["q"], s["k"] = (_normal(g, B, H, S, hd).to(t).transpose(1, 2) for H in (Hq, Hk))
            cut = rs.randint(0, S, size=B)  # two documents a sequence
            pos = np.stack([np.concatenate([np.arange(c), np.arange(S - c)]) for c in cut])
        s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        s["q_out"], s["k_out"] = (torch.empty_like(s[n]) for n in ("q", "k"))
    elif op == "plan":
        B, page = case["B"], case["page"]
        past, new = (np.array(v, dtype=np.int64) for v in _step(case))
        held = -(-past // page)
        need = np.where(new > 0, -(-(past + np.maximum(new, 0)) // page) - held, 0)
        n_pages = int(held.sum() + need.sum()) + 5
        perm = rs.permutation(n_pages).astype(np.int32)
        table = np.full((B, max(1, int((held + need).max()))), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += int(held[b])
        head = int(rs.randint(0, n_pages))
        free = n_pages - at
        ring = np.full(n_pages, -1, dtype=np.int32)
        ring[(head + np.arange(free)) % n_pages] = perm[at:]
        s["table"], s["ring"] = torch.from_numpy(table).cuda(), torch.from_numpy(ring).cuda()
        s["state"] = torch.tensor([head, free, 0, 0], dtype=I32, device="cuda")
        s["past"], s["new"] = (torch.from_numpy(v.astype(np.int32)).cuda() for v in (past, new))
        s["labels"] = torch.from_numpy(rs.randint(-1, 40, size=B).astype(np.int32)).cuda()
        M = int(np.maximum(new, 0).sum()) + case["pad"]
        s["M"] = M
        s["lens_out"], s["state_out"] = torch.empty_like(s["past"]), torch.empty_like(s["state"])
        s["slots"], s["positions"], s["owner"] = (torch.empty(M, dtype=I32, device="cuda") for _ in range(3))
        s["starts"] = torch.empty(B + 1, dtype=I32, device="cuda")
    else:
        N, k, n, R, L = (case[x] for x in ("N", "k", "n", "R", "L"))
        s["x"] = _normal(g, N, k).to(BF16)
        if case["wide"]:  # a slice of a fused projection's output
            s["y"] = _normal(g, N, 2 * n).to(BF16)[:, n:]
            s["out"] = torch.empty((N, 2 * n), dtype=BF16, device="cuda")[:, n:]
        else:
            s["y"] = _normal(g, N, n).to(BF16)
            s["out"] = torch.empty((N, n), dtype=BF16, device="cuda")
        s["a"] = (_normal(g, L, R, k) / math.sqrt(k)).to(BF16)
        s["b"] = (_normal(g, L, n, R) / math.sqrt(R)).to(BF16)
        s["scale"] = 0.5 + torch.rand(L, generator=g, device="cuda")
        s["ranks"] = torch.tensor(_ranks(case), dtype=I32, device="cuda") if case["ranks"] == "ragged" else None
        s["ids"] = torch.tensor(_ids(case), dtype=I32, device="cuda")
    if own:  # the handles that a program keeps beside its tensors
        from activation_sparse_ffn_gate_gb300 import binding
        s["lib"] = binding
        if op == "rope":
            s["rotary"] = binding.Rotary(s["freq"].cpu(), case["hd"], interleaved=case["pairs"] == "neighbours",
                                         factor=s["factor"], device=s["pos"].device)
        elif op == "plan":
            s["pool"] = binding.PagePool(s["ring"], s["state"], case["page"])
            s["plan"] = binding.StepPlan(s["slots"], s["positions"], s["owner"], s["starts"])
        else:
            s["adapters"] = binding.Adapters(s["a"], s["b"], s["scale"], s["ranks"])
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = s["pos"].to(F64)[..., None, None] * s["freq"]
    if c["way"] == "bwd":
        angle = -angle
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        t, rest = x[..., :rot], x[..., rot:]
        a, b = (t[..., :half], t[..., half:]) if c["pairs"] == "half" else (t[..., 0::2], t[..., 1::2])
        u, v = a * cos - b * sin, a * sin + b * cos
        t = torch.cat([u, v], -1) if c["pairs"] == "half" else torch.stack([u, v], -1).flatten(-2)
        out[name] = torch.cat([t, rest], -1).to(s[name].dtype)
    return out


def _plan(s):
    c = s["case"]
    page, B, M = c["page"], c["B"], s["M"]
    n = s["ring"].numel()
    head, free = s["state"][0].long(), s["state"][1].long()
    past, new = s["past"].long(), s["new"].long()
    add = new.clamp_min(0)
    ends = new == -1
    held = (past + page - 1) // page
    need = torch.where(add > 0, (past + add + page - 1) // page - held, 0)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    starts = torch.cat([zero, add.cumsum(0)])
    first = torch.cat([zero, need.cumsum(0)])  # of each request among the pages taken
    back = torch.where(ends, held, 0)
    gone = torch.cat([zero, back.cumsum(0)])
    table, ring = s["table"].clone(), s["ring"].clone()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, s["ring"][(head + first[:-1, None] + col - held[:, None]) % n], table)
    leaving = col < back[:, None]
    at = (head + free + gone[:-1, None] + col) % n
    spare = torch.full((1,), n, dtype=torch.int64, device="cuda")
    ring = torch.cat([ring, ring[:1]]).scatter(0, torch.where(leaving, at, spare).flatten(), table.flatten())[:n]
    i = torch.arange(M, device="cuda")
    b = torch.searchsorted(starts, i, right=True) - 1
    live = b < B
    b = b.clamp_max(B - 1)
    pos = past[b] + i - starts[b]
    pg = table[b, torch.where(live, pos // page, 0)]
    lens = torch.where(ends, 0, past + add)
    state = torch.stack([(head + first[-1]) % n, free - first[-1] + gone[-1], zero[0], zero[0]])
    return {"slots": torch.where(live, pg.long() * page + pos % page, -1).to(I32), "positions": torch.where(live, pos, 0).to(I32),
            "owner": torch.where(live, s["labels"][b].long(), -1).to(I32), "starts": starts.to(I32), "table": table,
            "lens": lens.to(I32), "ring": ring, "state": state.to(I32)}


def _lora(s):
    c = s["case"]
    N, L, R = c["N"], c["L"], c["R"]
    ids = s["ids"].long()
    t = (s["x"].float() @ s["a"].float().view(L * R, -1).t()).view(N, L, R) * s["scale"][:, None]
    use = (ids[:, None] == torch.arange(L, device="cuda"))[..., None]
    b = s["b"].float()
    if s["ranks"] is not None:
        low = torch.arange(R, device="cuda") < s["ranks"][:, None]
        use = use & low
    t = torch.where(use, t, 0.0).view(N, L * R)
    return {"y": (s["y"].float() + t @ b.transpose(1, 2).reshape(L * R, -1)).to(BF16)}


def run(s):
    op, c = s["op"], s["case"]
    if not own:
        return {"rope": _rope, "plan": _plan, "lora": _lora}[op](s)
    lib = s["lib"]
    if op == "rope":
        call = lib.twell_rope_fwd if c["way"] == "fwd" else lib.twell_rope_bwd
        q, k = call(s["q"], s["k"], s["pos"], s["rotary"], s["q_out"], s["k_out"])
        return {"q": q, "k": k}
    if op == "plan":
        p = lib.twell_kv_plan(s["pool"], s["table"], s["past"], s["new"], s["M"], labels=s["labels"], plan=s["plan"],
                              seq_lens_out=s["lens_out"], state_out=s["state_out"])
        return {"slots": p.slots, "positions": p.positions, "owner": p.owner, "starts": p.starts, "table": s["table"],
                "lens": s["lens_out"], "ring": s["ring"], "state": s["state_out"]}
    return {"y": lib.twell_lora_add(s["y"], s["x"], s["adapters"], s["ids"], out=s["out"])}


def work(case):
    op = case["op"]
    if op == "rope":
        N, H = case["B"] * case["S"], case["Hq"] + case["Hk"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * N * H * case["hd"] * e + 4 * N + 8 * (case["rot"] // 2), "flops": 3 * N * H * case["rot"]}
    if op == "plan":
        past, new = _step(case)
        page = case["page"]
        tokens = sum(max(v, 0) for v in new)
        pages = sum(-(-(p + max(v, 0)) // page) + -(-p // page) * (-1 if v >= 0 else 0) for p, v in zip(past, new))
        return {"bytes": 12 * (tokens + case["pad"]) + 8 * pages + 20 * case["B"], "flops": 4 * tokens}
    N, k, n = case["N"], case["k"], case["n"]
    ids, ranks = _ids(case), _ranks(case)
    used = sum(ranks[a] for a in set(ids) if a >= 0)
    turned = sum(1 for a in ids if a >= 0)
    return {"bytes": 2 * used * (k + n) + 2 * turned * k + 4 * N * n + 4 * N,
            "flops": 2 * (k + n) * sum(ranks[a] for a in ids if a >= 0)}


# ------------------------------------------------------------------------------------------ 64 bits

def _rope64(s):
    c = s["case"]
    rot = c["rot"]
    w = s["pos"].double()[..., None, None] * s["freq"] * (1 if c["way"] == "fwd" else -1)
    w = torch.polar(torch.full_like(w, s["factor"]), w)
    out = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        if c["pairs"] == "half":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * w
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * w
            x[..., :rot] = torch.view_as_real(z).flatten(-2)
        out[name] = x
    return out


def _plan64(s):
    """One request after the other, on the host."""
    c = s["case"]
    page, M, B = c["page"], s["M"], c["B"]
    old = s["ring"].cpu().numpy().astype(np.int64)
    table, ring, n = s["table"].cpu().numpy().astype(np.int64), old.copy(), len(old)
    head, free = (int(v) for v in s["state"][:2])
    tail = head + free
    past, new, labels = (s[x].cpu().tolist() for x in ("past", "new", "labels"))
    slots, positions, owner = np.full(M, -1), np.zeros(M, dtype=np.int64), np.full(M, -1)
    starts, lens, at = [], [], 0
    for b in range(B):
        starts.append(at)
        held = (past[b] + page - 1) // page
        if new[b] < 0:
            for p in range(held):
                ring[tail % n] = table[b, p]
                tail += 1
            lens.append(0)
            continue
        lens.append(past[b] + new[b])
        while held * page < lens[-1] and new[b] > 0:
            table[b, held] = old[head % n]
            held, head = held + 1, head + 1
        pos = np.arange(past[b], lens[-1])
        positions[at:at + new[b]] = pos
        slots[at:at + new[b]] = table[b, pos // page] * page + pos % page
        owner[at:at + new[b]] = labels[b]
        at += new[b]
    out = {"slots": slots, "positions": positions, "owner": owner, "starts": np.array(starts + [at]), "table": table,
           "lens": np.array(lens), "ring": ring, "state": np.array([head % n, tail - head, 0, 0])}
    return {name: torch.from_numpy(np.asarray(v, dtype=np.int64)).cuda() for name, v in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope64(s)
    if case["op"] == "plan":
        return _plan64(s)
    y = s["y"].double().clone()
    ids, ranks = np.array(_ids(case)), _ranks(case)
    for a in sorted(set(ids.tolist()) - {-1}):
        rows = torch.from_numpy(np.flatnonzero(ids == a)).cuda()
        A, Bm = s["a"][a, :ranks[a]].double(), s["b"][a, :, :ranks[a]].double()
        y[rows] += float(s["scale"][a]) * (s["x"][rows].double() @ A.t()) @ Bm.t()
    return {"y": y}
