"""The attention operators of a serving step, as measured cases.

Between the q/k/v projections and the o projection of a mixed multi-LoRA batch
a step builds its block tables and slot maps, rotates q and k, writes K and V
into a paged 4-bit cache, and attends: prompts over their own tokens, running
requests over the cache.  Each case is one pass through one of these; `run`
computes it with plain torch operations, or, where `own` is set, through the
framework's entry points.

Cache format (one layer): a block holds `bt` tokens; its bytes are records
[kv head][unit of 16 tokens] of 544*nc bytes, nc = head_dim/32:
  K codes [16 t][4 g][nc c][4 b]   nibbles: dims 32c+8g+2b (low), +1 (high) of token t
  V codes [4 g][16 d][nc c][4 j]   nibbles: dims 32c+d (low), 32c+16+d (high) of token 4g+j
  K scales [16 t][nc c], V scales [16 t][nc c]   2^(byte-127)
Codes are sign, 2 exponent bits and 1 fraction bit: 0 .5 1 1.5 2 3 4 6.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's bookkeeping: 1024 running requests, one new token each (the serving batch of the benchmark)
        dict(name="build_decode_1024", op="build", B=1024, lo=1, hi=4096, power=1.0, chunks=0, chunk=0, bt=16),
        # a step that admits many prompts next to running requests, contexts skewed to the short side
        dict(name="build_mixed_2000", op="build", B=2000, lo=1, hi=8192, power=3.0, chunks=64, chunk=2048, bt=64),
        # latency: one decode token of each of 16 requests, grouped heads
        dict(name="append_decode_16", op="append", T=16, hq=32, hkv=8, D=128, rot=128, half=True, scaling="none", dtype="bf16"),
        # the benchmark's decode batch: 1024 tokens, 32 heads of 128, context stretched by ramps between frequencies
        dict(name="append_decode_1024", op="append", T=1024, hq=32, hkv=32, D=128, rot=128, half=True, scaling="yarn", dtype="bf16"),
        # prompts of a prefill step, interleaved pairs, half of the head rotated
        dict(name="append_prompt_38781", op="append", T=38781, hq=32, hkv=8, D=128, rot=64, half=False, scaling="linear", dtype="bf16"),
        # latency: one request with a long context
        dict(name="attend_one_32k", op="attend", B=1, lo=32768, hi=32768, power=1.0, chunks=0, chunk=0, bt=16, hq=32, hkv=8, D=128, dtype="bf16"),
        # a small ordinary decode batch, ragged
        dict(name="attend_ragged_48", op="attend", B=48, lo=1, hi=2049, power=2.0, chunks=0, chunk=0, bt=16, hq=32, hkv=8, D=64, dtype="bf16"),
        # a large decode batch with as many kv heads as q heads
        dict(name="attend_decode_128", op="attend", B=128, lo=129, hi=4097, power=1.0, chunks=0, chunk=0, bt=32, hq=32, hkv=32, D=128, dtype="bf16"),
        # chunked prefill next to decode tokens: four requests bring 512 new tokens over their cached context
        dict(name="attend_mixed_64", op="attend", B=64, lo=100, hi=5000, power=2.0, chunks=4, chunk=512, bt=64, hq=32, hkv=8, D=128, dtype="bf16"),
        # latency: a short prompt of its own
        dict(name="prompt_one_211", op="prompt", B=1, lo=211, hi=211, power=1.0, hq=16, hkv=4, D=64, dtype="bf16"),
        # the prefill batch of the benchmark: 32 prompts of 128..2048 tokens
        dict(name="prompt_packed_32", op="prompt", B=32, lo=128, hi=2048, power=1.0, hq=32, hkv=32, D=128, dtype="bf16"),
        # long prompts next to a very short one
        dict(name="prompt_long_3", op="prompt", B=3, lo=1, hi=8192, power=1.0, hq=32, hkv=8, D=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["build", "append", "attend", "prompt"])
    hq, hkv = rng.choice([(32, 32), (32, 8), (16, 2), (8, 8), (20, 4), (40, 10), (28, 4), (32, 1)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    bt = rng.choice([16, 32, 64, 128])
    if op == "build":
        B = _log_int(rng, 1, 2000)
        return dict(op=op, B=B, lo=1, hi=_log_int(rng, 2, 8192), power=rng.uniform(0.5, 3.0),
                    chunks=rng.randint(0, min(B, 64)), chunk=_log_int(rng, 1, 2048), bt=bt)
    if op == "append":
        D = rng.choice([32, 64, 128, 160, 256])
        T = _log_int(rng, 1, int(1.0e9 / (D * (4 * (hq + hkv) + 6.2 * hkv))))
        return dict(op=op, T=T, hq=hq, hkv=hkv, D=D, rot=rng.choice([D, D // 2]), half=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    dtype="bf16" if T > 5000 else dtype)
    if op == "attend":
        D = rng.choice([64, 128, 160, 256])
        most = 128 * 2000 * 32 * 128 // (hkv * D)  # cached tokens of all requests
        hi = _log_int(rng, 1, 32768)
        B = _log_int(rng, 1, max(1, min(256, most // hi)))
        chunks = rng.choice([0, 0, rng.randint(0, min(B, 4))])
        return dict(op=op, B=B, lo=1 if B > 1 else hi, hi=hi, power=rng.uniform(0.5, 3.0), chunks=chunks,
                    chunk=_log_int(rng, 2, max(2, min(512, int(4e9) // (B * hi * hq)))) if chunks else 0, bt=bt, hq=hq, hkv=hkv, D=D, dtype=dtype)
    D = rng.choice([64, 128, 160, 256])
    hi = _log_int(rng, 1, min(8192, int(8192 * math.sqrt(4096 / (hq * D)))))
    B = _log_int(rng, 1, max(1, min(64, int(3.0e7 * 4096 / (hq * D)) // (hi * hi) or 1)))
    return dict(op=op, B=B, lo=1 if B > 1 else hi, hi=hi, power=rng.uniform(0.5, 2.0), hq=hq, hkv=hkv, D=D,
                dtype="bf16" if hi > 400 else dtype)


def _lengths(case):
    """Lengths after the step and new tokens of each request, in ascending order (the seed permutes them)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    u = [(i / (B - 1) if B > 1 else 1.0) ** case["power"] for i in range(B)]
    total = [lo + int(round((hi - lo) * x)) for x in u]
    n = case.get("chunks", 0)
    new = [1] * (B - n) + [min(t, case["chunk"]) for t in total[B - n:]]
    return total, new


def work(case):
    if case["op"] == "build":
        total, new = _lengths(case)
        T, bt = sum(new), case["bt"]
        blocks = sum(-(-t // bt) - -(-(t - n) // bt) for t, n in zip(total, new))
        # lengths in; table entries, slots, positions, owners, row offsets and lengths out
        return {"bytes": 4 * (2 * case["B"] + 2 * blocks + 3 * T + 2 * case["B"] + 1), "flops": 0}
    size = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "append":
        T, D, hq, hkv = case["T"], case["D"], case["hq"], case["hkv"]
        cached = T * hkv * 2 * (D // 2 + D // 32)
        # q, k, v in; q and the cached rows out; the cached rows read back as bf16 values
        moved = T * D * size * (2 * hq + 2 * hkv) + 2 * cached + T * D * hkv * 2 * 2
        return {"bytes": moved + T * 8, "flops": T * D * (hq + hkv) * 3}
    total, new = _lengths(case)
    D, hq, hkv = case["D"], case["hq"], case["hkv"]
    if case["op"] == "attend":
        cached = sum(total) * hkv * 2 * (D // 2 + D // 32)
        keys = sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(total, new))
        return {"bytes": cached + 2 * sum(new) * hq * D * size, "flops": 4 * keys * hq * D}
    keys = sum(t * (t + 1) // 2 for t in total)
    return {"bytes": sum(total) * D * size * (2 * hq + 2 * hkv), "flops": 4 * keys * hq * D}


# ------------------------------------------------------------------ the inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _frequencies(rot, scaling, theta=10000.0, factor=8.0, original=4096):
    """Radians per position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / max(rot - 2, 1))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        keep = 1.0 - np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    if scaling == "bands":
        turns = original * f / (2 * math.pi)
        mix = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f * mix + f / factor * (1.0 - mix), 1.0
    return f, 1.0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def _requests(case, seed):
    rng = np.random.default_rng(seed + 1)
    total, new = _lengths(case)
    order = rng.permutation(case["B"])
    return np.asarray(total, np.int64)[order], np.asarray(new, np.int64)[order], rng


def prepare(case, seed):
    s = dict(case)
    if case["op"] in ("build", "attend"):
        total, new, rng = _requests(case, seed)
        B, bt = case["B"], case["bt"]
        ctx = total - new
        have, need = -(-ctx // bt), -(-total // bt)
        blocks = int(need.sum())
        num_blocks = blocks + 5
        ids = rng.permutation(num_blocks)[:blocks].astype(np.int32)
        width = int(need.max()) + 3
        table = np.full((B, width), -1, np.int32)
        full = table.copy()
        at, free = 0, []
        for i in range(B):
            row = ids[at:at + need[i]]
            at += need[i]
            full[i, :need[i]] = row
            table[i, :have[i]] = row[:have[i]]
            free.append(row[have[i]:])
        s.update(ctx=_i32(ctx), new=_i32(new), T=int(new.sum()), num_blocks=num_blocks, free=_i32(np.concatenate(free)),
                 table=_i32(table if case["op"] == "build" else full), width=width, most_new=int(new.max()),
                 most=int(total.max()))
    if case["op"] == "append":
        T, D, g = case["T"], case["D"], _gen(seed)
        # the projections' output, k and v of a token side by side; positions of a long context; slots of a scattered cache
        q = torch.randn((T, case["hq"], D), generator=g, device=DEV).to(_dtype(case))
        k, v = torch.randn((T, 2 * case["hkv"], D), generator=g, device=DEV).to(_dtype(case)).split(case["hkv"], dim=1)
        rng = np.random.default_rng(seed + 1)
        bt, blocks = 16, -(-T // 16) + 3
        perm = rng.permutation(blocks)
        if T > 1024:  # prompts: neighbours in a block; a decode batch: each token in a block of its own request
            t = np.arange(T)
            slots, pos = perm[t // bt] * bt + t % bt, t % 2048
        else:
            blocks = T + 3
            slots = rng.permutation(blocks)[:T] * bt + rng.integers(0, bt, T)
            pos = rng.integers(0, 131072, T)
        freq, factor = _frequencies(case["rot"], case["scaling"])
        nc = D // 32
        s.update(q=q, k=k, v=v, q_out=torch.empty((T, case["hq"], D), dtype=_dtype(case), device=DEV),
                 slots=_i32(slots), pos=_i32(pos), freq=torch.tensor(freq, dtype=torch.float64, device=DEV), factor=factor, bt=bt,
                 cache=torch.zeros((blocks, case["hkv"] * 544 * nc), dtype=torch.uint8, device=DEV))
    if case["op"] == "attend":
        g, D, nc = _gen(seed), case["D"], case["D"] // 32
        records = case["hkv"] * case["bt"] // 16
        data = torch.empty((s["num_blocks"], records, 544 * nc), dtype=torch.uint8, device=DEV)
        borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        step = max(1, (1 << 27) // (records * 512 * nc))
        for a in range(0, s["num_blocks"], step):  # codes of normal values, scales that hold them
            part = data[a:a + step]
            x = torch.randn((part.shape[0], records, 512 * nc, 2), generator=g, device=DEV) * 2.3
            code = torch.bucketize(x.abs(), borders, out_int32=True) + 8 * (x < 0)
            part[..., :512 * nc] = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
            part[..., 512 * nc:] = torch.randint(125, 128, (part.shape[0], records, 32 * nc), generator=g, device=DEV, dtype=torch.uint8)
            del x, code
        s["cache"] = data.view(s["num_blocks"], -1)
        s["q"] = torch.randn((s["T"], case["hq"], D), generator=g, device=DEV).to(_dtype(case))
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "prompt":
        total, _, _ = _requests(case, seed)
        g, D, T = _gen(seed), case["D"], int(total.sum())
        q = torch.randn((T, case["hq"], D), generator=g, device=DEV).to(_dtype(case))
        k, v = torch.randn((T, 2 * case["hkv"], D), generator=g, device=DEV).to(_dtype(case)).split(case["hkv"], dim=1)
        s.update(T=T, most=int(total.max()), indptr=_i32(np.concatenate([[0], np.cumsum(total)])), q=q, k=k, v=v,
                 out=torch.empty((T, case["hq"], D), dtype=_dtype(case), device=DEV))
    return s


# ------------------------------------------------------------------ the framework's calls
def _handles(s):
    """The descriptors and workspaces that a serving program keeps between its steps (no values of the inputs)."""
    from heterogeneous_adapters_amd import kv
    h = {}
    if s["op"] == "build":
        h["batch"] = kv.Batch(s["T"], s["B"], 8, 8, 128)
    if s["op"] == "append":
        h["cache"] = kv.Cache(s["cache"], s["bt"], s["hkv"], s["D"])
        h["rope"] = kv.Rope(s["freq"], kv.ROPE_HALF if s["half"] else kv.ROPE_INTERLEAVED, s["factor"])
        h["k"] = torch.empty((s["T"], s["hkv"], s["D"]), dtype=torch.bfloat16, device=DEV)
        h["v"] = torch.empty_like(h["k"])
    if s["op"] == "attend":
        h["cache"] = kv.Cache(s["cache"], s["bt"], s["hkv"], s["D"])
        h["batch"] = kv.Batch(s["T"], s["B"], s["hq"], s["hkv"], s["D"])
        h["ws"] = kv.attend_workspace(h["batch"])
    return kv, h


def _run_own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    kv, h = s["handles"]
    if s["op"] == "append":
        kv.lora_kv_append(s["q"], s["q_out"], s["k"], s["v"], s["pos"], s["slots"], h["rope"], h["cache"])
        kv.lora_kv_gather(h["cache"], s["slots"], h["k"], h["v"])
        return {"q": s["q_out"], "k": h["k"], "v": h["v"]}
    if s["op"] == "prompt":
        kv.lora_prompt_attend(s["q"], s["k"], s["v"], s["out"], s["indptr"], 1.0 / math.sqrt(s["D"]))
        return s["out"]
    b = h["batch"]
    kv.lora_kv_build(s["ctx"], s["new"], s["T"], s["table"], s["free"], s["num_blocks"], s["bt"], b)
    if s["op"] == "build":
        return {"table": s["table"], "q_indptr": b.q_indptr, "kv_len": b.kv_len, "seq": b.token_seq, "pos": b.positions,
                "slots": b.slots, "used": b.new_blocks}
    kv.lora_kv_attend(s["q"], s["out"], b, s["table"], h["cache"], 1.0 / math.sqrt(s["D"]), h["ws"])
    return s["out"]


# ------------------------------------------------------------------ the plain forms
def _plain_build(s):
    B, bt, T = s["B"], s["bt"], s["T"]
    ctx, new = s["ctx"].long(), s["new"].long()
    total = ctx + new
    end = new.cumsum(0)
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(end, t, right=True)
    pos = ctx[seq] + t - (end - new)[seq]
    have, need = (ctx + bt - 1) // bt, (total + bt - 1) // bt
    taken = (need - have).cumsum(0) - (need - have)
    col = torch.arange(s["width"], device=DEV)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (taken[:, None] + col - have[:, None]).clamp(0, max(s["free"].numel() - 1, 0))
    ids = s["free"][at] if s["free"].numel() else s["table"]
    table = torch.where(fresh, ids, s["table"])
    slots = table[seq, pos // bt] * bt + (pos % bt).int()
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    return {"table": table, "q_indptr": torch.cat([zero, end]).int(), "kv_len": total.int(), "seq": seq.int(), "pos": pos.int(),
            "slots": slots.int(), "used": (need - have).sum().int().view(1)}


def _plain_rotate(x, pos, freq, factor, rot, half):
    # angles of far positions, and keys that are rounded to a few bits afterwards: in 64 bits
    a = pos.double()[:, None, None] * freq
    c, n = a.cos() * factor, a.sin() * factor
    r = x[..., :rot].double()
    one, two = (r[..., :rot // 2], r[..., rot // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    u, w = one * c - two * n, two * c + one * n
    r = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([r.to(x.dtype), x[..., rot:]], -1)


def _plain_four_bits(x):
    """Values of groups of 32 in sign, 2 exponent bits and 1 fraction bit, with the smallest power of two whose sevenfold holds them."""
    g = x.float().unflatten(-1, (-1, 32))
    most = g.abs().amax(-1, keepdim=True)
    frac, e = torch.frexp(most)  # most = frac * 2^e, frac in [.5, 1)
    e = torch.where(frac > 0.875, e - 2, e - 3).clamp(min=-95)
    y = torch.ldexp(g, -e)
    m = y.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)  # halves go to the even multiple
    return torch.ldexp(torch.where(y < 0, -m, m), e).flatten(-2).to(torch.bfloat16)


def _plain_append(s):
    q = _plain_rotate(s["q"], s["pos"], s["freq"], s["factor"], s["rot"], s["half"])
    k = _plain_rotate(s["k"], s["pos"], s["freq"], s["factor"], s["rot"], s["half"])
    return {"q": q, "k": _plain_four_bits(k), "v": _plain_four_bits(s["v"])}


def _plain_values(codes):
    m = (codes & 7).int()
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.where(codes >= 8, -lut[m], lut[m])


def _plain_cache(s):
    """K and V of every request, padded to the longest: [B, L, hkv, D]."""
    B, H, D, nc, bt = s["B"], s["hkv"], s["D"], s["D"] // 32, s["bt"]
    nb, U = -(-s["most"] // bt), bt // 16
    rec = s["cache"][s["table"][:, :nb].clamp(min=0).long()].view(B, nb, H, U, 544 * nc)
    kc, vc, ks, vs = rec.split([256 * nc, 256 * nc, 16 * nc, 16 * nc], dim=-1)
    scale = lambda x: torch.ldexp(torch.ones((), device=DEV), x.int() - 127).view(B, nb, H, U, 16, nc)  # noqa: E731
    k = _plain_values(torch.stack([kc & 15, kc >> 4], -1)).view(B, nb, H, U, 16, 4, nc, 4, 2)
    k = k.permute(0, 1, 3, 4, 2, 6, 5, 7, 8).reshape(B, nb, U, 16, H, nc, 32) * scale(ks).permute(0, 1, 3, 4, 2, 5)[..., None]
    v = _plain_values(torch.stack([vc & 15, vc >> 4], -1)).view(B, nb, H, U, 4, 16, nc, 4, 2)
    v = v.permute(0, 1, 3, 4, 7, 2, 6, 8, 5).reshape(B, nb, U, 16, H, nc, 32) * scale(vs).permute(0, 1, 3, 4, 2, 5)[..., None]
    return k.reshape(B, nb * bt, H, D), v.reshape(B, nb * bt, H, D)


def _plain_softmax(x, seen):
    x = torch.where(seen, x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-38)


def _plain_attend(s):
    B, H, D, G, N = s["B"], s["hkv"], s["D"], s["hq"] // s["hkv"], s["most_new"]
    k, v = _plain_cache(s)
    L = k.shape[1]
    new, ctx = s["new"].long(), s["ctx"].long()
    start = new.cumsum(0) - new
    j = torch.arange(N, device=DEV)
    row = (start[:, None] + j).clamp(max=s["T"] - 1)  # [B, N]: rows behind a request's last are computed and dropped
    q = s["q"].float()[row].view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(B, H, G, N, L) * (1.0 / math.sqrt(D))
    pos = ctx[:, None] + j
    seen = torch.arange(L, device=DEV) <= pos[..., None]
    p = _plain_softmax(x, seen[:, None, None])
    o = torch.matmul(p.view(B, H, G * N, L), v.permute(0, 2, 1, 3).contiguous())
    o = o.view(B, H, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, H * G, D)
    return o[j[None, :] < new[:, None]].to(s["q"].dtype)


def _plain_prompt(s):
    B, H, D, G, L, T = s["B"], s["hkv"], s["D"], s["hq"] // s["hkv"], s["most"], s["T"]
    start, n = s["indptr"][:-1].long(), (s["indptr"][1:] - s["indptr"][:-1]).long()
    j = torch.arange(L, device=DEV)
    row = (start[:, None] + j).clamp(max=T - 1)
    q = s["q"].float()[row].view(B, L, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * L, D)
    k = s["k"].float()[row].permute(0, 2, 3, 1).contiguous()
    v = s["v"].float()[row].permute(0, 2, 1, 3).contiguous()
    x = torch.matmul(q, k).view(B, H, G, L, L) * (1.0 / math.sqrt(D))
    p = _plain_softmax(x, j[None, :] <= j[:, None])
    o = torch.matmul(p.view(B, H, G * L, L), v).view(B, H, G, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, H * G, D)
    return o[j[None, :] < n[:, None]].to(s["q"].dtype)


def run(s):
    if own:
        return _run_own(s)
    return {"build": _plain_build, "append": _plain_append, "attend": _plain_attend, "prompt": _plain_prompt}[s["op"]](s)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_rows(q, k, v, first, D):
    """Softmax attention of rows q [n, hq, D] at positions first.. over k, v [L, hkv, D], in pieces of rows."""
    n, hq, _ = q.shape
    L, hkv, _ = k.shape
    out = torch.empty((n, hq, D), dtype=torch.float64, device=DEV)
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        last = min(L, first + b)  # keys behind the piece's last position are seen by none of its rows
        hide = torch.arange(last, device=DEV)[None, :] > torch.arange(first + a, first + b, device=DEV)[:, None]
        for h in range(hkv):
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            w = q[a:b, mine].double().transpose(0, 1) @ k[:last, h].double().T.contiguous() / D ** 0.5
            w = w.masked_fill(hide, -math.inf)
            w = torch.exp(w - w.max(dim=2, keepdim=True).values)
            out[a:b, mine] = ((w @ v[:last, h].double()) / w.sum(dim=2, keepdim=True)).transpose(0, 1)
    return out


def exact(case, seed):
    if case["op"] == "build":
        return None  # whole numbers, compared as such
    s = prepare(case, seed)
    D = case["D"]
    if case["op"] == "append":
        a = s["pos"].double().view(-1, 1) * s["freq"].view(1, -1)
        z = torch.polar(torch.full_like(a, s["factor"]), a)[:, None, :]  # pairs as complex numbers, turned
        q, rot = s["q"].double(), case["rot"]
        i = torch.arange(rot // 2, device=DEV)
        re, im = (i, i + rot // 2) if case["half"] else (2 * i, 2 * i + 1)
        turned = torch.complex(q[..., re].contiguous(), q[..., im].contiguous()) * z
        q[..., re], q[..., im] = turned.real, turned.imag
        return {"q": q, "k": None, "v": None}  # what is held in 4 bits has no nearer value than the one of its code
    if case["op"] == "prompt":
        at = s["indptr"].tolist()
        return torch.cat([_exact_rows(s["q"][a:b], s["k"][a:b], s["v"][a:b], 0, D) for a, b in zip(at, at[1:])])
    # attend: the byte of each (token, dim), by the format's formulas
    bt, nc, H = case["bt"], D // 32, case["hkv"]
    t, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    c, r = d // 32, d % 32
    k_at, k_high = ((t * 4 + r // 8) * nc + c) * 4 + (r % 8) // 2, r % 2
    v_at, v_high = 256 * nc + (((t // 4) * 16 + r % 16) * nc + c) * 4 + t % 4, r // 16
    ks_at, vs_at = 512 * nc + t * nc + c, 528 * nc + t * nc + c
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)

    def read(rec, at, high, sc):
        code = (rec[..., at] >> (4 * high).to(torch.uint8)) & 15
        return value[code.long()] * torch.pow(2.0, rec[..., sc].double() - 127.0)

    got, begin = [], 0
    for i, (ctx, new) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        L = ctx + new
        rec = s["cache"][s["table"][i, :-(-L // bt)].long()].view(-1, H, bt // 16, 544 * nc).transpose(1, 2).reshape(-1, H, 544 * nc)
        k = read(rec, k_at, k_high, ks_at).transpose(1, 2).reshape(-1, H, D)[:L]
        v = read(rec, v_at, v_high, vs_at).transpose(1, 2).reshape(-1, H, D)[:L]
        got.append(_exact_rows(s["q"][begin:begin + new], k, v, ctx, D))
        begin += new
    return torch.cat(got)
