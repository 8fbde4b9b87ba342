"""Shared prompts and beam search over the paged 4-bit cache, as measured cases.

Requests that begin with the same tokens (a system prompt in front of every
request of an adapter, the beams of one request) attend to that prefix
together: `shared` builds a step's batch and its shared plan and attends.
Beams are chosen from the step's logits (`select`); the survivors then take
over their parents' block tables, and blocks that two of them would write to
are copied in every layer's cache (`reorder`).  Each case is one pass through
one of these; `run` computes it with plain torch operations, or, where `own`
is set, through the framework's entry points.

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
        # latency: the four beams of one request over its prompt
        dict(name="shared_beams_4", op="shared", B=4, groups=1, plo=1000, phi=1000, lo=1, hi=120, chunks=0, chunk=0, bt=16,
             hq=32, hkv=8, D=128, dtype="bf16"),
        # a small ordinary decode batch: adapters with system prompts of their own, some requests without
        dict(name="shared_ragged_48", op="shared", B=48, groups=6, plo=200, phi=2500, lo=1, hi=700, chunks=0, chunk=0, bt=16,
             hq=32, hkv=8, D=64, dtype="bf16"),
        # as many kv heads as q heads: a row of its own for every request
        dict(name="shared_mha_96", op="shared", B=96, groups=8, plo=256, phi=4096, lo=1, hi=600, chunks=0, chunk=0, bt=32,
             hq=32, hkv=32, D=128, dtype="bf16"),
        # a large decode batch behind one long document
        dict(name="shared_decode_256", op="shared", B=256, groups=1, plo=32768, phi=32768, lo=1, hi=500, chunks=0, chunk=0,
             bt=64, hq=32, hkv=8, D=128, dtype="bf16"),
        # four requests bring 512 new tokens next to decode tokens, all behind two prompts
        dict(name="shared_chunks_32", op="shared", B=32, groups=2, plo=3000, phi=6000, lo=1, hi=900, chunks=4, chunk=512, bt=64,
             hq=32, hkv=8, D=128, dtype="bf16"),
        # latency: one request of four beams
        dict(name="select_1x4", op="select", B=1, W=4, V=32000, done=0.0, alpha=0.0, dtype="bf16"),
        # an odd vocabulary in 32 bits, scores by length
        dict(name="select_32x5", op="select", B=32, W=5, V=50257, done=0.1, alpha=0.6, dtype="f32"),
        # a large batch and vocabulary
        dict(name="select_64x8", op="select", B=64, W=8, V=128000, done=0.05, alpha=1.0, dtype="bf16"),
        # the most rows
        dict(name="select_128x16", op="select", B=128, W=16, V=32000, done=0.1, alpha=0.0, dtype="bf16"),
        # latency: one request of four beams, a few layers
        dict(name="reorder_1x4", op="reorder", B=1, W=4, plo=500, phi=500, hi=77, bt=16, hkv=8, D=128, layers=4),
        # many requests of eight beams, blocks of 64 tokens
        dict(name="reorder_96x8", op="reorder", B=96, W=8, plo=30, phi=2000, hi=300, bt=64, hkv=8, D=128, layers=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "select", "reorder"])
    if op == "select":
        W, V = rng.randint(1, 16), _log_int(rng, 1000, 160000)
        return dict(op=op, B=_log_int(rng, 1, max(1, int(6.5e7 / (W * V)))), W=W, V=V, done=rng.choice([0.0, 0.1, 0.3]),
                    alpha=rng.choice([0.0, 0.6, 1.0, -0.5]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    bt = rng.choice([16, 32, 64, 128])
    if op == "reorder":
        hkv, D, W = rng.choice([1, 4, 8]), rng.choice([64, 96, 128]), rng.randint(1, 12)
        return dict(op=op, B=_log_int(rng, 1, max(1, 90 * 8 * 16 // (W * max(bt, 16)))), W=W, plo=1, phi=_log_int(rng, 1, 2000), hi=_log_int(rng, 1, 300),
                    bt=bt, hkv=hkv, D=D, layers=rng.randint(1, 4))
    hq, hkv = rng.choice([(32, 32), (32, 8), (16, 2), (8, 8), (20, 4), (40, 10), (28, 4), (32, 1)])
    D = rng.choice([64, 128, 160, 256])
    phi = _log_int(rng, 16, 32768)
    B = _log_int(rng, 1, max(1, min(256, int(256 * 32768 * 32 * 128 / (phi * hq * D)))))
    groups = rng.randint(1, max(1, min(B, 16, 200000 // phi, 40000 * 8 * 128 // (phi * hkv * D))))
    hi = _log_int(rng, 1, min(600, max(2, 150000 * 8 * 128 // (B * hkv * D))))
    chunks = rng.choice([0, 0, rng.randint(0, min(B, 4))])
    most = max(2, min(512, int(2e9 / (hq * B * (hi + 512))), int(256 * 32768 / (5 * phi))))
    return dict(op=op, B=B, groups=groups, plo=max(1, phi // 8), phi=phi, lo=1, hi=hi, chunks=chunks,
                chunk=_log_int(rng, 2, most) if chunks else 0, bt=bt, hq=hq, hkv=hkv, D=D, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))


def _spread(lo, hi, n, i):
    return lo + int(round((hi - lo) * (i / (n - 1) if n > 1 else 1.0)))


def _shared_lengths(case):
    """Group of each request (-1: none), shared tokens of each group (whole blocks), tokens of its own that a request
    has cached, and new ones."""
    B, n, bt = case["B"], case["groups"], case["bt"]
    alone = B // 12 if n > 1 else 0  # requests with a prompt of their own, at the end
    group = [i * n // (B - alone) for i in range(B - alone)] + [-1] * alone
    prefix = [max(_spread(case["plo"], case["phi"], n, g) // bt * bt, bt) for g in range(n)]
    mine = [_spread(case["lo"], case["hi"], B, (i * 7919) % B) - 1 for i in range(B)]
    k = case["chunks"]
    new = [case["chunk"] if k and i % (B // k) == 0 and i // (B // k) < k else 1 for i in range(B)]
    return group, prefix, mine, new


def _beam_lengths(case):
    """Prompt and generated tokens of each request."""
    B = case["B"]
    prompt = [_spread(case["plo"], case["phi"], B, i) for i in range(B)]
    return prompt, [_spread(1, case["hi"], B, (i * 7919) % B) for i in range(B)]


def work(case):
    if case["op"] == "select":
        rows = case["B"] * case["W"]
        return {"bytes": rows * (case["V"] * (2 if case["dtype"] == "bf16" else 4) + 32), "flops": 0}
    record = 17 * case["D"]  # bytes of 16 tokens of a kv head
    if case["op"] == "reorder":
        prompt, made = _beam_lengths(case)
        B, W, bt = case["B"], case["W"], case["bt"]
        table = sum(-(-(p + m) // bt) for p, m in zip(prompt, made)) * W * 4 * 2
        # on average over random parents a share (1 - 1/W)^W of the beams leave nobody, as many blocks are copied
        units = sum(-(-((p + m) % bt) // 16) for p, m in zip(prompt, made)) * W * (1 - 1 / W) ** W
        return {"bytes": table + B * W * 12 + int(2 * units * case["hkv"] * record * case["layers"]), "flops": 0}
    group, prefix, mine, new = _shared_lengths(case)
    size = 2 if case["dtype"] == "bf16" else 4
    have = sum(prefix) + sum(m + n for m, n in zip(mine, new))
    keys = sum(n * ((prefix[g] if g >= 0 else 0) + m) + n * (n + 1) // 2 for g, m, n in zip(group, mine, new))
    return {"bytes": have * case["hkv"] * record // 16 + 2 * sum(new) * case["hq"] * case["D"] * size,
            "flops": 4 * keys * case["hq"] * case["D"]}


# ------------------------------------------------------------------ the inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def _prepare_shared(case, seed, s):
    g, rng = _gen(seed), np.random.default_rng(seed + 1)
    B, bt, H, nc = case["B"], case["bt"], case["hkv"], case["D"] // 32
    group, prefix, mine, new = _shared_lengths(case)
    own_at = np.asarray([prefix[i] if i >= 0 else 0 for i in group])  # where a request's own tokens begin
    ctx, new = own_at + np.asarray(mine), np.asarray(new)
    total = ctx + new
    have, need, lead = -(-ctx // bt), -(-total // bt), own_at // bt
    blocks = int(sum(p // bt for p in prefix) + (need - lead).sum())
    num_blocks, width = blocks + 5, int(need.max()) + 3
    ids, at = rng.permutation(num_blocks)[:blocks].astype(np.int32), 0
    shared_ids = []
    for p in prefix:
        shared_ids.append(ids[at:at + p // bt])
        at += p // bt
    table, free = np.full((B, width), -1, np.int32), []
    for i in range(B):
        row = ids[at:at + need[i] - lead[i]]
        at += need[i] - lead[i]
        if group[i] >= 0:
            table[i, :lead[i]] = shared_ids[group[i]]
        table[i, lead[i]:need[i]] = row
        free.append(row[have[i] - lead[i]:])
    indptr = np.searchsorted(np.asarray([x if x >= 0 else case["groups"] for x in group]), np.arange(case["groups"] + 1))
    # codes of normal values, scales that hold them
    records = H * bt // 16
    data = torch.empty((num_blocks, records, 544 * nc), dtype=torch.uint8, device=DEV)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = max(1, (1 << 27) // (records * 512 * nc))
    for a in range(0, num_blocks, step):
        part = data[a:a + step]
        x = torch.randn((part.shape[0], records, 512 * nc, 2), generator=g, device=DEV) * 2.3
        code = torch.bucketize(x.abs(), borders, out_int32=True) + 8 * (x < 0)
        part[..., :512 * nc] = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
        part[..., 512 * nc:] = torch.randint(125, 128, (part.shape[0], records, 32 * nc), generator=g, device=DEV, dtype=torch.uint8)
        del x, code
    T = int(new.sum())
    q = torch.randn((T, case["hq"], case["D"]), generator=g, device=DEV).to(_dtype(case))
    s.update(T=T, num_blocks=num_blocks, ctx=_i32(ctx), new=_i32(new), table=_i32(table), free=_i32(np.concatenate(free)),
             indptr=_i32(indptr), shared_len=_i32(prefix), cache=data.view(num_blocks, -1), q=q, out=torch.empty_like(q),
             # what the plain form's loops run over, on the host
             h_indptr=indptr.tolist(), h_prefix=list(prefix), h_own=own_at.tolist(), h_ctx=ctx.tolist(), h_new=new.tolist())


def _prepare_select(case, seed, s):
    g = _gen(seed)
    B, W, V = case["B"], case["W"], case["V"]
    # the beams of a request see much the same text
    logits = torch.randn((B, 1, V), generator=g, device=DEV) * 2.5 + torch.randn((B, W, V), generator=g, device=DEV) * 0.7
    score = -(torch.rand((B, W), generator=g, device=DEV) * 2).cumsum(1) - 3
    length = torch.randint(3, 60, (B, W), generator=g, device=DEV, dtype=torch.int32)
    done = (torch.rand((B, W), generator=g, device=DEV) < case["done"]).int()
    empty = lambda t: torch.empty(B * W, dtype=t, device=DEV)  # noqa: E731
    s.update(logits=logits.view(B * W, V).to(_dtype(case)), score=score.flatten(), length=length.flatten(), done_in=done.flatten(), eos=V - 3,
             out={"parent": empty(torch.int32), "token": empty(torch.int32), "score": empty(torch.float32),
                  "length": empty(torch.int32), "done": empty(torch.int32)})


def _prepare_reorder(case, seed, s):
    g, rng = _gen(seed), np.random.default_rng(seed + 1)
    B, W, bt, H, nc = case["B"], case["W"], case["bt"], case["hkv"], case["D"] // 32
    prompt, made = _beam_lengths(case)
    lens = [p + m for p, m in zip(prompt, made)]
    width = -(-max(lens) // bt) + 2
    table, used = np.full((B * W, width), -1, np.int32), 0
    for b in range(B):  # beams share a block up to where their lines of descent part
        last = -(-lens[b] // bt)
        line = np.arange(W)
        for j in range(last - 1, -1, -1):
            if j < prompt[b] // bt:
                line = np.zeros(W, np.int64)
            elif j < last - 1:
                line = np.sort(rng.integers(0, W, W))[line]
            names, mine = np.unique(line, return_inverse=True)
            table[b * W:(b + 1) * W, j] = used + mine
            used += len(names)
    # as many blocks as beams that share none of what they generated would fill
    num_blocks = sum(p // bt + W * (-(-n // bt) - p // bt) for p, n in zip(prompt, lens)) + B * W + 7
    ids = rng.permutation(num_blocks).astype(np.int32)
    table = np.where(table >= 0, ids[table], -1)
    parent = (rng.integers(0, W, (B, W)) + np.arange(B)[:, None] * W).reshape(-1)
    bytes_ = H * (bt // 16) * 544 * nc
    caches = [torch.randint(0, 256, (num_blocks, bytes_), generator=g, device=DEV, dtype=torch.uint8) for _ in range(case["layers"])]
    R = B * W
    minus = lambda *n: torch.full(n, -1, dtype=torch.int32, device=DEV)  # noqa: E731
    s.update(parent=_i32(parent), kv_len=_i32(np.repeat(lens, W)), table=_i32(table), free=_i32(ids[used:used + R]), num_blocks=num_blocks,
             caches=caches, new_table=minus(R, width), new_len=minus(R))


def prepare(case, seed):
    s = dict(case)
    {"shared": _prepare_shared, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, seed, s)
    return s


# ------------------------------------------------------------------ the framework's calls
def _handles(s):
    """The descriptors and workspaces that a serving program keeps between its steps (no values of the inputs)."""
    from heterogeneous_adapters_amd import beam, kv
    h = {}
    if s["op"] == "shared":
        h["cache"] = kv.Cache(s["cache"], s["bt"], s["hkv"], s["D"])
        h["batch"] = kv.Batch(s["T"], s["B"], s["hq"], s["hkv"], s["D"])
        h["shared"] = kv.Shared(h["batch"], s["groups"])
        h["ws"] = kv.shared_workspace(h["batch"], h["shared"])
    if s["op"] == "select":
        h["ws"] = beam.select_workspace(s["B"], s["W"], s["V"])
        h["beams"] = beam.Beams(s["score"], s["length"], s["done_in"])
        h["next"] = beam.Beams(s["out"]["score"], s["out"]["length"], s["out"]["done"])
    if s["op"] == "reorder":
        h["layers"] = beam.Layers([kv.Cache(c, s["bt"], s["hkv"], s["D"]) for c in s["caches"]])
        h["moves"] = beam.Moves(s["B"] * s["W"], s["table"].shape[1])
        h["moves"].freed.fill_(-1)
    return kv, beam, h


def _run_own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    kv, beam, h = s["handles"]
    if s["op"] == "shared":
        b = h["batch"]
        kv.lora_kv_build(s["ctx"], s["new"], s["T"], s["table"], s["free"], s["num_blocks"], s["bt"], b)
        kv.lora_kv_share(s["indptr"], s["shared_len"], b, h["shared"])
        kv.lora_kv_attend_shared(s["q"], s["out"], b, h["shared"], s["table"], h["cache"], 1.0 / math.sqrt(s["D"]), h["ws"])
        return s["out"]
    if s["op"] == "select":
        out = s["out"]
        beam.lora_beam_select(s["logits"], s["W"], h["beams"], out["parent"], out["token"], h["next"], h["ws"],
                              length_penalty=s["alpha"], eos=s["eos"])
        return out
    m = h["moves"]
    beam.lora_beam_reorder(s["parent"], s["W"], s["kv_len"], s["table"], s["new_len"], s["new_table"], s["free"], s["num_blocks"],
                           s["bt"], m)
    beam.lora_beam_copy(m, h["layers"])
    return {"table": s["new_table"], "kv_len": s["new_len"], "source": m.source, "target": m.target, "tokens": m.tokens,
            "freed": m.freed, "copies": m.copies, "given_back": m.given_back, "caches": s["caches"]}


# ------------------------------------------------------------------ the plain forms
def _plain_values(codes):
    m = (codes & 7).int()
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.where(codes >= 8, -lut[m], lut[m])


def _plain_blocks(s, ids):
    """K and V of blocks ids [n, nb]: [n, nb * bt, kv heads, D]."""
    H, D, nc, bt = s["hkv"], s["D"], s["D"] // 32, s["bt"]
    n, nb = ids.shape
    rec = s["cache"][ids.clamp(min=0).long()].view(n, nb, H, bt // 16, 544 * nc)
    kc, vc, ks, vs = rec.split([256 * nc, 256 * nc, 16 * nc, 16 * nc], dim=-1)
    scale = lambda x: torch.ldexp(torch.ones((), device=DEV), x.int() - 127).view(n, nb, H, bt // 16, 16, nc)  # noqa: E731
    k = _plain_values(torch.stack([kc & 15, kc >> 4], -1)).view(n, nb, H, bt // 16, 16, 4, nc, 4, 2)
    k = k.permute(0, 1, 3, 4, 2, 6, 5, 7, 8).reshape(n, nb, bt // 16, 16, H, nc, 32) * scale(ks).permute(0, 1, 3, 4, 2, 5)[..., None]
    v = _plain_values(torch.stack([vc & 15, vc >> 4], -1)).view(n, nb, H, bt // 16, 4, 16, nc, 4, 2)
    v = v.permute(0, 1, 3, 4, 7, 2, 6, 8, 5).reshape(n, nb, bt // 16, 16, H, nc, 32) * scale(vs).permute(0, 1, 3, 4, 2, 5)[..., None]
    return k.reshape(n, nb * bt, H, D), v.reshape(n, nb * bt, H, D)


def _plain_shared(s):
    """The prefix of a group by one product for all of its rows; what is a request's own, padded to the longest."""
    B, H, D, G, bt, T = s["B"], s["hkv"], s["D"], s["hq"] // s["hkv"], s["bt"], s["T"]
    N, norm = max(s["h_new"]), 1.0 / math.sqrt(s["D"])
    new, ctx = s["new"].long(), s["ctx"].long()
    start = new.cumsum(0) - new
    j = torch.arange(N, device=DEV)
    live = j[None, :] < new[:, None]
    own_at = torch.tensor(s["h_own"], device=DEV)
    nb = max(-(-(c + n - o) // bt) for c, n, o in zip(s["h_ctx"], s["h_new"], s["h_own"]))
    col = own_at[:, None] // bt + torch.arange(nb, device=DEV)
    k, v = _plain_blocks(s, s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)))
    L = nb * bt
    row = (start[:, None] + j).clamp(max=T - 1)  # rows behind a request's last are computed and dropped
    q = s["q"].float()[row].view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(B, H, G, N, L) * norm
    seen = own_at[:, None, None] + torch.arange(L, device=DEV) <= (ctx[:, None] + j)[..., None]
    x = torch.where(seen[:, None, None], x, -math.inf)
    most = x.amax(-1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, G * N, L), v.permute(0, 2, 1, 3).contiguous()).view(B, H, G, N, D)
    flat = lambda y: y.permute(0, 3, 1, 2, 4).reshape(B * N, H, G, -1)[live.view(-1)]  # noqa: E731
    most, total, o = flat(most), flat(total), flat(o)  # [T, H, G, 1 or D]
    out = o / total
    for a, b, p in zip(s["h_indptr"], s["h_indptr"][1:], s["h_prefix"]):
        k, v = _plain_blocks(s, s["table"][a:a + 1, :p // bt])
        t0 = sum(s["h_new"][:a])
        t1 = t0 + sum(s["h_new"][a:b])
        q = s["q"][t0:t1].float().view(t1 - t0, H, G, D).permute(1, 2, 0, 3).reshape(H, -1, D)
        x = torch.matmul(q, k[0].permute(1, 2, 0).contiguous()) * norm  # [H, rows, p]
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        y = torch.matmul(e, v[0].transpose(0, 1).contiguous())
        back = lambda w: w.view(H, G, t1 - t0, -1).permute(2, 0, 1, 3)  # noqa: E731
        m, z, y = back(m), back(z), back(y)
        top = torch.maximum(m, most[t0:t1])
        u, w = torch.exp(m - top), torch.exp(most[t0:t1] - top)
        out[t0:t1] = (y * u + o[t0:t1] * w) / (z * u + total[t0:t1] * w)
    return out.reshape(T, H * G, D).to(s["q"].dtype)


def _plain_select(s):
    # scores next to one another decide which beams live: in 64 bits
    B, W, V, R = s["B"], s["W"], s["V"], s["B"] * s["W"]
    x = s["logits"].double()
    most = x.amax(-1, keepdim=True)
    x = x - most
    x -= torch.exp(x).sum(-1, keepdim=True).log()
    x += s["score"].double()[:, None]
    done = s["done_in"] != 0
    # a finished beam stands for itself alone
    x[done] = -math.inf
    x[:, 0] = torch.where(done, s["score"].double(), x[:, 0])
    length = torch.where(done, s["length"], s["length"] + 1)
    if s["alpha"] != 0.0:
        x /= length.clamp(min=1).double()[:, None] ** s["alpha"]
    x = x.view(B, W * V)
    at = []
    for _ in range(W):
        at.append(x.argmax(-1, keepdim=True))  # the lowest of equal ones
        x.scatter_(1, at[-1], -math.inf)
    at = torch.cat(at, 1)
    parent = (at // V + torch.arange(B, device=DEV)[:, None] * W).view(R)
    kept = done[parent]
    token = torch.where(kept, s["eos"], (at % V).view(R))
    line = s["logits"].double()[parent]
    gain = line.gather(1, token[:, None])[:, 0] - line.amax(-1)
    gain -= torch.exp(line - line.amax(-1, keepdim=True)).sum(-1).log()
    score = s["score"].double()[parent] + torch.where(kept, 0.0, gain)
    return {"parent": parent.int(), "token": token.int(), "score": score.float(), "length": length[parent],
            "done": (kept | (token == s["eos"])).int()}


def _plain_reorder(s):
    B, W, bt, R = s["B"], s["W"], s["bt"], s["B"] * s["W"]
    table, width = s["table"], s["table"].shape[1]
    p, free = s["parent"].long(), s["free"]
    n = s["kv_len"].long()[p]
    blocks, col = (n + bt - 1) // bt, torch.arange(width, device=DEV)
    out = torch.where(col < blocks[:, None], table[p], -1)
    kin = p.view(B, W)
    older = (kin[:, :, None] == kin[:, None, :]).tril(-1).any(-1).view(R)  # an earlier beam has the same parent
    need = older & (n % bt != 0)
    rows = need.nonzero()[:, 0]
    at = n[rows] // bt
    source, target, tokens = table[p[rows], at], free[:rows.numel()], (n[rows] % bt).int()
    out[rows, at] = target
    # blocks that no beam holds any longer, each once
    old = (s["kv_len"].long()[:, None] + bt - 1) // bt > col
    t, o = table.view(B, W, width), old.view(B, W, width)
    kt, ko = table[p].view(B, W, width), (col < blocks[:, None]).view(B, W, width)
    held = ((t[:, :, None] == kt[:, None]) & ko[:, None]).any(2)
    again = torch.stack([((t[:, :r] == t[:, r:r + 1]) & o[:, :r]).any(1) for r in range(W)], 1)
    gone = (o & ~held & ~again).transpose(1, 2)  # by request, column, row
    freed = t.transpose(1, 2)[gone]
    pad = lambda x, m: torch.cat([x, torch.full((m - x.numel(),), -1, dtype=torch.int32, device=DEV)])  # noqa: E731
    count = lambda x: torch.full((1,), x.numel(), dtype=torch.int32, device=DEV)  # noqa: E731
    units = torch.arange(bt // 16, device=DEV)
    fill = (units * 16 < tokens[:, None])[:, None, :, None]  # whole units of 16 tokens
    for c in s["caches"]:
        v = c.view(c.shape[0], s["hkv"], bt // 16, -1)
        v[target.long()] = torch.where(fill, v[source.long()], v[target.long()])
    return {"table": out, "kv_len": n.int(), "source": pad(source, R), "target": pad(target, R), "tokens": pad(tokens, R),
            "freed": pad(freed, R * width), "copies": count(source), "given_back": count(freed), "caches": s["caches"]}


def run(s):
    if own:
        return _run_own(s)
    return {"shared": _plain_shared, "select": _plain_select, "reorder": _plain_reorder}[s["op"]](s)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_rows(q, k, v, first, D):
    """Softmax attention of rows q [n, hq, D] at positions first.. over k, v [L, hkv, D], in pieces of rows."""
    n, hq, _ = q.shape
    L, hkv, _ = k.shape
    out = torch.empty((n, hq, D), dtype=torch.float64, device=DEV)
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        hide = torch.arange(L, device=DEV)[None, :] > torch.arange(first + a, first + b, device=DEV)[:, None]
        for h in range(hkv):
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            w = q[a:b, mine].double().transpose(0, 1) @ k[:, h].double().T.contiguous() / D ** 0.5
            w = w.masked_fill(hide, -math.inf)
            w = torch.exp(w - w.max(dim=2, keepdim=True).values)
            out[a:b, mine] = ((w @ v[:, h].double()) / w.sum(dim=2, keepdim=True)).transpose(0, 1)
    return out


def _exact_shared(s):
    """Every request by itself, over its own table row; the byte of each (token, dim) by the format's formulas."""
    D, bt, nc, H = s["D"], s["bt"], s["D"] // 32, s["hkv"]
    t, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    c, r = d // 32, d % 32
    k_at, k_high = ((t * 4 + r // 8) * nc + c) * 4 + (r % 8) // 2, r % 2
    v_at, v_high = 256 * nc + (((t // 4) * 16 + r % 16) * nc + c) * 4 + t % 4, r // 16
    ks_at, vs_at = 512 * nc + t * nc + c, 528 * nc + t * nc + c
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)

    def read(rec, at, high, sc):
        code = (rec[..., at] >> (4 * high).to(torch.uint8)) & 15
        return value[code.long()] * torch.pow(2.0, rec[..., sc].float() - 127.0)  # exact in 32 bits

    got, begin = [], 0
    for i, (ctx, new) in enumerate(zip(s["h_ctx"], s["h_new"])):
        L = ctx + new
        rec = s["cache"][s["table"][i, :-(-L // bt)].long()].view(-1, H, bt // 16, 544 * nc).transpose(1, 2).reshape(-1, H, 544 * nc)
        k = read(rec, k_at, k_high, ks_at).transpose(1, 2).reshape(-1, H, D)[:L]
        v = read(rec, v_at, v_high, vs_at).transpose(1, 2).reshape(-1, H, D)[:L]
        got.append(_exact_rows(s["q"][begin:begin + new], k, v, ctx, D))
        begin += new
    return torch.cat(got)


def exact(case, seed):
    if case["op"] == "reorder":
        return None  # whole numbers, compared as such
    s = prepare(case, seed)
    if case["op"] == "shared":
        return _exact_shared(s)
    # every request's candidates sorted; which are chosen are whole numbers, their scores are not
    B, W, V = case["B"], case["W"], case["V"]
    score = torch.empty(B, W, dtype=torch.float64, device=DEV)
    for b in range(B):
        p = torch.softmax(s["logits"][b * W:(b + 1) * W].double(), -1)
        total = p.log() + s["score"][b * W:(b + 1) * W, None]
        length = s["length"][b * W:(b + 1) * W, None] + 1
        done = s["done_in"][b * W:(b + 1) * W].bool()
        rank = total / length.double().pow(case["alpha"])
        alone, kept = s["score"][b * W:(b + 1) * W].double()[done], s["length"][b * W:(b + 1) * W].double()[done]
        value = torch.cat([alone, total[~done].flatten()])
        order = torch.cat([alone / kept.pow(case["alpha"]), rank[~done].flatten()]).topk(W).indices
        score[b] = value[order]
    return {"parent": None, "token": None, "score": score.flatten(), "length": None, "done": None}
