"""Cases of the operators around the shared cache: page tables, the 4-bit cache, retention.

Four operators of one serving step of a YOCO model:

* ``tables``  block tables extended and token slots worked out from request lengths
* ``append``  new K/V rows quantised to 4 bits (e2m1, one power-of-two scale for 32 head dims)
              into cache pages through the slots, and those rows read back
* ``attend``  causal paged GQA attention over the 4-bit cache, a step's layers with one plan
* ``retain``  linear attention with a decay per head: prompts in chunks, single tokens recurrently

``run`` computes them in elementary torch operations, or with ``own`` through the library.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step's bookkeeping: 64 running requests, one token each
        dict(name="tables, 64 decoding", op="tables", decode=64, prefill=0, lo=1024, hi=8192, block=16),
        # a busy mixed step: many short requests decoding, a few prompts admitted
        dict(name="tables, 1500 and 12 prompts", op="tables", decode=1500, prefill=12, lo=17, hi=4099, block=32),
        # the decode step's new rows: one token per request
        dict(name="append, 64 tokens", op="append", tokens=64, kv_heads=2, dim=256, block=16),
        # a prefill step's rows (the mixed workload's count)
        dict(name="append, 23900 tokens", op="append", tokens=23900, kv_heads=2, dim=256, block=16),
        # a small service: three requests with short, ragged contexts
        dict(name="attend, 3 short", op="attend", reqs=3, lo=1, hi=301, rows=1, q_heads=8, kv_heads=2, dim=128, block=16, layers=2),
        # pure decode at the workload's shapes
        dict(name="attend, 64 decoding", op="attend", reqs=64, lo=1024, hi=8192, rows=1, q_heads=8, kv_heads=2, dim=256, block=16, layers=4),
        # long contexts, one kv head for all queries
        dict(name="attend, 4 of 131072", op="attend", reqs=4, lo=131072, hi=131072, rows=1, q_heads=16, kv_heads=1, dim=128, block=32, layers=4),
        # speculative verification: four rows of each request
        dict(name="attend, 64 x 4 rows", op="attend", reqs=64, lo=1028, hi=8196, rows=4, q_heads=8, kv_heads=2, dim=256, block=16, layers=2),
        # single tokens, decay by token, a few streams
        dict(name="retain, 5 decoding", op="retain", decode=5, prefill=0, lo=1, hi=1, q_heads=8, kv_heads=8, dim=128, gated=True),
        # single tokens of a full batch
        dict(name="retain, 64 decoding", op="retain", decode=64, prefill=0, lo=1, hi=1, q_heads=8, kv_heads=8, dim=256, gated=True),
        # a mixed step: prompts admitted while others decode
        dict(name="retain, 16 and 4 prompts", op="retain", decode=16, prefill=4, lo=1024, hi=4096, q_heads=8, kv_heads=8, dim=256, gated=True),
        # one long prompt, fixed decays, shared k/v heads
        dict(name="retain, one of 16384", op="retain", decode=0, prefill=1, lo=16384, hi=16384, q_heads=8, kv_heads=2, dim=128, gated=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "retain", "retain"])
    if op == "tables":
        lo = _log(rng, 1, 2048)
        return dict(op=op, decode=_log(rng, 1, 1500), prefill=rng.randint(0, 12), lo=lo, hi=lo + _log(rng, 1, 2048),
                    block=rng.choice([16, 32]))
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 23900), kv_heads=rng.choice([1, 2]), dim=rng.choice([128, 256]),
                    block=rng.choice([16, 32]))
    if op == "attend":
        kv = rng.choice([1, 2])
        group = rng.choice([1, 3, 4, 8, 16])
        reqs = _log(rng, 1, 64)
        lo = _log(rng, 1, 4096)
        hi = lo + _log(rng, 1, min(4096, max(2, 131072 // reqs)))
        return dict(op=op, reqs=reqs, lo=lo, hi=hi, rows=rng.choice([1, 1, 2, 3]), q_heads=group * kv, kv_heads=kv,
                    dim=rng.choice([128, 256]), block=rng.choice([16, 32]), layers=rng.choice([1, 2, 3]))
    kv = rng.choice([1, 2, 4])
    decode = _log(rng, 1, 64)
    prefill = rng.choice([0, 1, 2, 3])
    lo = _log(rng, 2, 2048)
    return dict(op=op, decode=decode, prefill=prefill, lo=lo, hi=lo + _log(rng, 1, 1024), q_heads=kv * rng.choice([1, 2]),
                kv_heads=kv, dim=rng.choice([64, 128, 256]), gated=rng.choice([True, False]))


# ------------------------------------------------- the 4-bit format, plainly
#
# A code is sign, two exponent bits, one mantissa bit; 32 consecutive head
# dims of a token share the scale 2^(b - 127), the smallest with every
# magnitude at most 6 of it (b within [1, 251]).

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# magnitudes half way between two levels go to the even code
MIDDLES = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def _encode(x):
    """[..., D] -> codes uint8 [..., D] and scale bytes uint8 [..., D / 32]."""
    g = x.float().unflatten(-1, (-1, 32))
    m, e = torch.frexp(g.abs().amax(-1))  # m in [0.5, 1): 6 * 2^s >= m * 2^e
    b = torch.where(m > 0, (e - 3 + (m > 0.75).int() + 127).clamp(1, 251), 1)
    y = torch.ldexp(g, (127 - b).unsqueeze(-1))
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, mid in enumerate(MIDDLES):
        code += (a > mid) if i % 2 == 0 else (a >= mid)
    code += 8 * torch.signbit(y).to(torch.uint8)
    return code.flatten(-2), b.to(torch.uint8)


def _pack(code):
    c = code.unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4)


def _decode(packed, b):
    """Packed codes [..., D / 2] and scale bytes [..., D / 32] -> float32 values."""
    table = torch.tensor(LEVELS + [-v for v in LEVELS], device=packed.device)
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    return torch.ldexp(table[code].unflatten(-1, (-1, 32)), (b.int() - 127).unsqueeze(-1)).flatten(-2)


# ----------------------------------------------------------------- prepare


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _lengths(g, n, lo, hi):
    """n lengths spread evenly over [lo, hi], in an order of the seed."""
    spread = lo + torch.round((hi - lo) * (torch.arange(n) + 0.5) / max(n, 1)).long()
    return spread[torch.randperm(n, generator=g)]


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    dev = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend,
            "retain": _prepare_retain}[case["op"]](s, host, dev)


def _prepare_tables(s, host, dev):
    R, bs = s["decode"] + s["prefill"], s["block"]
    seq = torch.cat([_lengths(host, n, s["lo"], s["hi"]) for n in (s["decode"], s["prefill"])])
    q = torch.ones(R, dtype=torch.int64)
    q[s["decode"]:] = seq[s["decode"]:]
    order = torch.randperm(R, generator=host)
    seq, q = seq[order], q[order]
    held, need = (seq - q + bs - 1) // bs, (seq + bs - 1) // bs
    width = int(s["hi"] + bs - 1) // bs + 1
    used, new = int(held.sum()), int((need - held).sum())
    num_blocks = int(1.2 * (used + new)) + 8
    perm = torch.randperm(num_blocks, generator=host)
    table = torch.full((R, width), -1, dtype=torch.int64)
    table[torch.arange(width) < held[:, None]] = perm[:used]
    free = perm[used:]
    qsl = torch.cat((torch.zeros(1, dtype=torch.int64), q.cumsum(0)))
    s.update(num_blocks=num_blocks, block_table=_i32(table), seq_lens=_i32(seq), qsl=_i32(qsl), free_pages=_i32(free),
             num_free=_i32([free.numel()]), num_free_after=_i32([0]), slots=_i32([0] * int(qsl[-1])),
             err=_i32([0]), tokens=int(qsl[-1]))
    return s


def _pools(num_blocks, s, fill=0):
    shape = (num_blocks, s["kv_heads"], s["block"], s["dim"] // 2)
    k = torch.full(shape, fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((num_blocks, s["kv_heads"], 2, s["block"], s["dim"] // 32), 127, dtype=torch.uint8, device="cuda")
    return k, k.clone(), scales


def _prepare_append(s, host, dev):
    T, H, D, bs = s["tokens"], s["kv_heads"], s["dim"], s["block"]
    # runs of consecutive slots in pages of any order, as a step's prompts and single tokens have them
    num_blocks = int(1.2 * T / bs) + 8
    pages = torch.randperm(num_blocks, generator=host)[: (T + bs - 1) // bs]
    slots = (pages[:, None] * bs + torch.arange(bs)).flatten()[:T]
    k, v, sc = _pools(num_blocks, s)
    new = [torch.randn(T, H, D, generator=dev, device="cuda").bfloat16() for _ in range(2)]
    s.update(slots=_i32(slots), k_cache=k, v_cache=v, scales=sc, k_new=new[0], v_new=new[1], err=_i32([0]),
             k_out=torch.empty_like(new[0]), v_out=torch.empty_like(new[1]))
    return s


def _prepare_attend(s, host, dev):
    R, K, bs, D, H = s["reqs"], s["rows"], s["block"], s["dim"], s["kv_heads"]
    seq = _lengths(host, R, s["lo"], s["hi"])
    need = (seq + bs - 1) // bs
    width = int(need.max())
    num_blocks = int(1.2 * int(need.sum())) + 4
    perm = torch.randperm(num_blocks, generator=host)
    table = torch.full((R, width), -1, dtype=torch.int64)
    table[torch.arange(width) < need[:, None]] = perm[: int(need.sum())]
    k, v, sc = _pools(num_blocks, s)
    step = max(1, (1 << 26) // (H * bs * D))
    for pool, which in ((k, 0), (v, 1)):
        for at in range(0, num_blocks, step):
            n = min(step, num_blocks - at)
            code, b = _encode(torch.randn(n, H, bs, D, generator=dev, device="cuda").bfloat16())
            pool[at:at + n] = _pack(code)
            sc[at:at + n, :, which] = b
    q = torch.randn(s["layers"], R * K, s["q_heads"], D, generator=dev, device="cuda").bfloat16()
    s.update(num_blocks=num_blocks, block_table=_i32(table), seq_lens=_i32(seq), cqsl=_i32(torch.arange(R + 1) * K), q=q,
             out=torch.empty_like(q), k_cache=k, v_cache=v, scales=sc, longest=int(seq.max()), err=_i32([0]),
             softmax_scale=D ** -0.5, kept={})
    return s


def _prepare_retain(s, host, dev):
    R, D, H, Hkv = s["decode"] + s["prefill"], s["dim"], s["q_heads"], s["kv_heads"]
    q_len = torch.ones(R, dtype=torch.int64)
    q_len[s["decode"]:] = _lengths(host, s["prefill"], s["lo"], s["hi"])
    before = torch.randint(1, 4096, (R,), generator=host)
    before[s["decode"]::2] = 0  # every other prompt is a new sequence, the others go on
    T = int(q_len.sum())
    num_states = R + 3
    where = torch.randperm(num_states, generator=host)[:R]
    randn = lambda *n: torch.randn(*n, generator=dev, device="cuda")  # noqa: E731
    if s["gated"]:  # a gate of each token and head: sigmoid(x)^(1/16)
        decay = torch.nn.functional.logsigmoid(randn(T, H)) / 16
    else:
        decay = torch.log1p(-torch.exp2(-5.0 - torch.arange(H, device="cuda"))).float()
    state = randn(num_states, H, D, D)
    s.update(q=randn(T, H, D).bfloat16(), k=(randn(T, Hkv, D) * D ** -0.5).bfloat16(), v=randn(T, Hkv, D).bfloat16(), decay=decay,
             state=state, after=state.clone(), where=_i32(where), qsl=_i32([0] + q_len.cumsum(0).tolist()),
             seq_lens=_i32(before + q_len), longest=int(q_len.max()), softmax_scale=D ** -0.5, err=_i32([0]), kept={}, tokens=T)
    s["out"] = torch.empty_like(s["q"])
    return s


# --------------------------------------------------------------------- run


def run(s):
    if own:
        return {"tables": _own_tables, "append": _own_append, "attend": _own_attend, "retain": _own_retain}[s["op"]](s)
    return {"tables": _tables, "append": _append, "attend": _attend, "retain": _retain}[s["op"]](s)


def _own_tables(s):
    from yoco_shared_kv_gb300 import _native as Y
    Y.yoco_build_block_tables(s["block_table"], s["seq_lens"], s["qsl"], s["num_blocks"], s["block"], s["slots"],
                              s["free_pages"], s["num_free"], s["num_free_after"], s["err"])
    return {"block_table": s["block_table"], "slots": s["slots"], "num_free": s["num_free_after"]}


def _own_append(s):
    from yoco_shared_kv_gb300 import _native as Y
    Y.yoco_kv_append_e2m1(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["scales"], s["slots"], s["err"])
    Y.yoco_kv_gather_e2m1(s["k_cache"], s["v_cache"], s["scales"], s["slots"], s["k_out"], s["v_out"], s["err"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attend(s):
    from yoco_shared_kv_gb300 import _native as Y
    R, K = s["reqs"], s["rows"]
    if "workspace" not in s["kept"]:
        n = Y.yoco_cross_attn_workspace_size(R * K, s["q_heads"], s["kv_heads"], s["dim"], s["block"], s["longest"], Y.E2M1)
        s["kept"]["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    ws = s["kept"]["workspace"]
    Y.yoco_cross_attn_plan(s["block_table"], s["seq_lens"], s["cqsl"], s["longest"], R * K, s["q_heads"], s["kv_heads"],
                           s["dim"], s["block"], s["num_blocks"], Y.E2M1, ws, s["err"])
    for layer in range(s["layers"]):
        flags = Y.YOCO_ATTN_PLANNED | (Y.YOCO_ATTN_OVERLAP if layer else 0) | (Y.YOCO_ATTN_REVERSE if layer % 2 else 0)
        Y.yoco_cross_attn_paged_e2m1(s["q"][layer], s["k_cache"], s["v_cache"], s["scales"], s["out"][layer], s["block_table"],
                                     s["seq_lens"], s["cqsl"], s["longest"], s["softmax_scale"], ws, s["err"], flags=flags)
    return s["out"]


def _own_retain(s):
    from yoco_shared_kv_gb300 import _native as Y
    if "workspace" not in s["kept"]:
        n = Y.yoco_retention_workspace_size(s["decode"] + s["prefill"], s["tokens"], s["longest"], s["q_heads"], s["dim"])
        s["kept"]["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    Y.yoco_retention(s["q"], s["k"], s["v"], s["decay"], s["state"], s["where"], s["out"], s["qsl"], s["seq_lens"], s["longest"],
                     s["softmax_scale"], s["kept"]["workspace"], s["after"], s["err"])
    return {"out": s["out"], "state": s["after"]}


def _tables(s):
    bs, seq, qsl = s["block"], s["seq_lens"].long(), s["qsl"].long()
    q = qsl[1:] - qsl[:-1]
    held, need = (seq - q + bs - 1) // bs, (seq + bs - 1) // bs
    end = (need - held).cumsum(0)
    lp = torch.arange(s["block_table"].shape[1], device="cuda")
    new = (lp >= held[:, None]) & (lp < need[:, None])
    nth = (end - need)[:, None] + lp  # how many pages were taken before this one
    taken = s["free_pages"].long()[(s["num_free"].long() - 1 - nth).clamp(0, s["free_pages"].numel() - 1)]
    table = torch.where(new, taken, s["block_table"].long())
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(qsl, t, right=True) - 1
    pos = seq[r] - q[r] + t - qsl[r]
    slots = table[r, pos // bs] * bs + pos % bs
    return {"block_table": table.int(), "slots": slots.int(), "num_free": (s["num_free"] - end[-1:]).int()}


def _append(s):
    page, at = s["slots"].long() // s["block"], s["slots"].long() % s["block"]
    got = {}
    for which, name in enumerate("kv"):
        code, b = _encode(s[name + "_new"])
        pool, scales = s[name + "_cache"], s["scales"][:, :, which]
        pool[page, :, at] = _pack(code)
        scales[page, :, at] = b
        got[name] = _decode(pool[page, :, at], scales[page, :, at]).bfloat16()
    return got


def _attend(s):
    R, K, bs, D, H = s["reqs"], s["rows"], s["block"], s["dim"], s["kv_heads"]
    G, layers = s["q_heads"] // H, s["layers"]
    page = s["block_table"].long().clamp(min=0)
    k, v = (_decode(pool[page], s["scales"][page, :, i]).transpose(1, 2).reshape(R, H, -1, D)
            for i, pool in enumerate((s["k_cache"], s["v_cache"])))
    # queries of a kv head together: [R, H, layers * K * G, D]
    q = s["q"].float().view(layers, R, K, H, G, D).permute(1, 3, 0, 2, 4, 5).reshape(R, H, -1, D)
    score = torch.matmul(q, k.transpose(2, 3)).mul_(s["softmax_scale"]).view(R, H, layers, K, G, -1)
    keys = s["seq_lens"].long()[:, None] - K + 1 + torch.arange(K, device="cuda")  # of each row
    seen = (torch.arange(k.shape[2], device="cuda") < keys[:, :, None]).view(R, 1, 1, K, 1, -1)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 4), v).view(R, H, layers, K, G, D) / torch.where(total == 0, 1.0, total)
    return o.permute(2, 0, 3, 1, 4, 5).reshape(layers, R * K, H * G, D).bfloat16()


def _padded(s):
    """Each request's tokens side by side: index [R, longest] and which of them are there."""
    qsl = s["qsl"].long()
    t = torch.arange(s["longest"], device="cuda")
    there = t < (qsl[1:] - qsl[:-1])[:, None]
    return torch.where(there, qsl[:-1, None] + t, 0), there


def _retain(s):
    H, G = s["q_heads"], s["q_heads"] // s["kv_heads"]
    at, there = _padded(s)
    live = there[:, :, None, None]
    q = torch.where(live, s["q"][at].float(), 0.0).transpose(1, 2)  # [R, H, L, D]
    k, v = (torch.where(live, s[n][at].float(), 0.0).transpose(1, 2).repeat_interleave(G, 1) for n in "kv")
    g = s["decay"].double().expand(s["tokens"], H)[at]
    c = torch.where(there[:, :, None], g, 0.0).cumsum(1).transpose(1, 2)  # [R, H, L]
    old = torch.where((s["seq_lens"] > s["qsl"][1:] - s["qsl"][:-1])[:, None, None, None], s["state"][s["where"].long()], 0.0)
    w = (c[..., :, None] - c[..., None, :]).float().exp_().tril_()
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)).mul_(w), v) + c.float().exp()[..., None] * torch.matmul(q, old)
    out = (o * s["softmax_scale"]).transpose(1, 2)[there].bfloat16()
    last = (c[..., -1:] - c).float().exp()[..., None]
    after = s["after"].clone()
    after[s["where"].long()] = c[..., -1:, None].float().exp() * old + torch.matmul(k.transpose(2, 3), v * last)
    return {"out": out, "state": after}


# -------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    mean = (case.get("lo", 0) + case.get("hi", 0)) / 2
    if op == "tables":
        R = case["decode"] + case["prefill"]
        tokens = case["decode"] + case["prefill"] * mean
        new = case["decode"] / case["block"] + case["prefill"] * (mean / case["block"] + 0.5)
        # lengths and offsets, one table entry a decoding request, free pages; entries and slots out
        return {"bytes": 8 * R + 4 * case["decode"] + 8 * new + 4 * tokens, "flops": 0}
    if op == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        # rows in, codes and scales out; those read again, rows out
        return {"bytes": n * (2 + 17 / 32 + 17 / 32 + 2) + 4 * case["tokens"], "flops": 0}
    if op == "attend":
        rows, D = case["reqs"] * case["rows"], case["dim"]
        keys = case["reqs"] * mean
        return {"bytes": case["layers"] * (keys * 2 * case["kv_heads"] * D * 17 / 32 + 4 * rows * case["q_heads"] * D),
                "flops": case["layers"] * 4 * keys * case["rows"] * case["q_heads"] * D}
    D, H = case["dim"], case["q_heads"]
    tokens = case["decode"] + case["prefill"] * mean
    rows = 2 * tokens * (2 * H + 2 * case["kv_heads"]) * D
    fresh = (case["prefill"] + 1) // 2  # new sequences read no state
    states = 4 * H * D * D * (2 * (case["decode"] + case["prefill"]) - fresh)
    return {"bytes": rows + states + 4 * H * (tokens if case["gated"] else 1), "flops": 4 * tokens * H * D * D}


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": lambda _: None, "append": _exact_append, "attend": _exact_attend, "retain": _exact_retain}[case["op"]](s)


def _exact_values(packed, b):
    """Values of packed codes in 64 bits, by the format's arithmetic."""
    n = torch.stack((packed.long() % 16, packed.long() // 16), -1).flatten(-2)
    e, m = n // 2 % 4, (n % 2).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    x = torch.where(n >= 8, -mag, mag).unflatten(-1, (-1, 32))
    return (x * torch.exp2(b.double() - 127)[..., None]).flatten(-2)


def _exact_append(s):
    got = {}
    levels = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    for name in "kv":
        x = s[name + "_new"].double().unflatten(-1, (-1, 32))
        top = x.abs().amax(-1, keepdim=True)
        unit = torch.exp2(torch.ceil(torch.log2((top / 6).clamp(min=2.0 ** -126))).clamp(-126, 124))
        a = (x / unit).abs()
        i = torch.searchsorted(levels, a).clamp(1, 7)
        low, high = levels[i - 1], levels[i]
        up = (a - low > high - a) | ((a - low == high - a) & (i % 2 == 0))
        got[name] = (torch.where(up, high, low) * torch.sign(x) * unit).flatten(-2)
    return got


def _exact_attend(s):
    H, D, bs, K = s["kv_heads"], s["dim"], s["block"], s["rows"]
    G = s["q_heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["seq_lens"].tolist()):
        pages = s["block_table"][r, : (n + bs - 1) // bs].long()
        for h in range(H):
            k, v = (_exact_values(pool[pages, h], s["scales"][pages, h, i]).reshape(-1, D)
                    for i, pool in enumerate((s["k_cache"], s["v_cache"])))
            for i in range(K):
                keys = n - K + i + 1
                if keys > 0:
                    q = s["q"][:, r * K + i, h * G:(h + 1) * G].double()
                    p = torch.softmax(q @ k[:keys].T * s["softmax_scale"], -1)
                    out[:, r * K + i, h * G:(h + 1) * G] = p @ v[:keys]
    return out


def _exact_retain(s):
    H, G, D = s["q_heads"], s["q_heads"] // s["kv_heads"], s["dim"]
    out = torch.zeros(s["tokens"], H, D, dtype=torch.float64, device="cuda")
    after = s["after"].double()
    ends = s["qsl"].tolist()
    for r in range(len(ends) - 1):
        a, b = ends[r], ends[r + 1]
        state = s["state"][s["where"][r].long()].double() * float(s["seq_lens"][r] > b - a)
        for t in range(a, b, 256):  # pieces short enough for products of decays
            u = min(t + 256, b)
            q = s["q"][t:u].double().transpose(0, 1)
            k, v = (s[n][t:u].double().transpose(0, 1).repeat_interleave(G, 0) for n in "kv")
            c = s["decay"].double().expand(s["tokens"], H)[t:u].T.cumsum(1)
            low = torch.ones(u - t, u - t, dtype=torch.bool, device="cuda").tril()
            w = torch.where(low, torch.exp(c[:, :, None] - c[:, None, :]), 0.0)
            o = (q @ k.transpose(1, 2) * w) @ v + torch.exp(c)[:, :, None] * (q @ state)
            out[t:u] = (o * s["softmax_scale"]).transpose(0, 1)
            w = torch.exp(c[:, -1:] - c)[:, :, None]
            state = torch.exp(c[:, -1])[:, None, None] * state + (k * w).transpose(1, 2) @ v
        after[s["where"][r].long()] = state
    return {"out": out, "state": after}
