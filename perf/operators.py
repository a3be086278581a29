"""The serving path's operators, measured one by one: the page step (block tables and slot maps from request
lengths), rotary positions (and their gradient), the rotary write into a paged cache, and differential attention of
new tokens over that cache.

``run`` makes the framework's calls where ``own`` is true and computes the same in elementary torch operations where
it is false; ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
LAMBDA_INIT = 0.5


# ---------------------------------------------------------------- the cases --
def listed():
    return [
        # one generated token for each of 64 requests of 1K to 32K tokens: every step of a decode loop
        dict(name="step-decode-64", op="step", S=64, page=64, ctx_lo=1024, ctx_hi=32767, new_hi=1, p_chunk=0.0,
             p_done=0.0, pad=0, lens=1),
        # a busy server's step: single tokens, chunks of prompts and finished requests, small pages
        dict(name="step-mixed-700", op="step", S=700, page=16, ctx_lo=0, ctx_hi=32767, new_hi=512, p_chunk=0.25,
             p_done=0.06, pad=77, lens=2),
        # a training batch (4 sequences of 4096, 12 heads): queries and keys before the attention
        dict(name="rope-train-bf16", op="rope", seqs=4, n=4096, H=12, Hkv=12, d=128, rot=128, layout="interleaved",
             dtype="bf16", inverse=False, kind="none", factor=1.0, pos_hi=4096),
        # the same step's backward: float32 gradients of packed sequences, half the head rotated, a long-context table
        dict(name="rope-grad-f32", op="rope", seqs=7, n=1171, H=20, Hkv=20, d=128, rot=64, layout="half",
             dtype="f32", inverse=True, kind="yarn", factor=8.0, pos_hi=32768),
        # the cache write of a decode step: 64 tokens, one per request
        dict(name="append-decode-64", op="append", T=64, pad=0, H=12, Hkv=12, d=128, rot=128, layout="interleaved",
             kind="linear", factor=4.0, page=64, pages=128, pos_hi=32768),
        # the cache write of a chunked step with shared key heads, pages of 16 and a padded batch
        dict(name="append-chunk-6001", op="append", T=6001, pad=143, H=20, Hkv=4, d=128, rot=64, layout="half",
             kind="ntk", factor=4.0, page=16, pages=700, pos_hi=65536),
        # the first tokens of one short request: latency alone
        dict(name="extend-one-77", op="extend", H=2, Hkv=2, d=64, page=16, causal=True, pad=0,
             new="1", kv="77", lens=0),
        # a decode step: 64 requests of 1K to 32K tokens, 12 heads (12.7 GB of keys and values)
        dict(name="extend-decode-64", op="extend", H=12, Hkv=12, d=128, page=64, causal=True, pad=0,
             S=64, new_lo=1, new_hi=1, kv_lo=1024, kv_hi=32768, lens=3),
        # drafted tokens to be checked: 5 for each of 24 requests
        dict(name="extend-verify-24x5", op="extend", H=16, Hkv=16, d=128, page=16, causal=True, pad=8,
             S=24, new_lo=5, new_hi=5, kv_lo=500, kv_hi=9001, lens=4),
        # a mixed step with shared key heads: single tokens beside chunks of two prompts
        dict(name="extend-mixed-20over4", op="extend", H=20, Hkv=4, d=128, page=32, causal=True, pad=13,
             new="1 1 1 1 1 1 1 1 1 1 1 1 301 33",
             kv="782 1559 2336 3113 3890 4667 5444 6221 6998 7775 8552 9329 4321 8190", lens=0),
        # a chunk of 2048 tokens behind 30K cached ones: a long prompt run through in chunks
        dict(name="extend-chunk-2048", op="extend", H=12, Hkv=12, d=128, page=64, causal=True, pad=0,
             new="2048", kv="32100", lens=0),
        # ragged prompts from an empty cache, narrow heads
        dict(name="extend-prompts-6", op="extend", H=16, Hkv=16, d=64, page=128, causal=True, pad=3,
             new="4000 1 129 640 1023 2048", kv="4000 1 129 640 1023 2048", lens=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "rope", "append", "extend", "extend", "extend"])
    d = rng.choice([64, 128])
    group = rng.choice([1, 1, 1, 2, 4, 5, 7])
    Hkv = rng.randint(1, max(1, 20 // group))
    kind = rng.choice(["none", "linear", "ntk", "yarn"])
    rope = dict(d=d, rot=rng.choice([d, d // 2, d // 4, d - 16]), layout=rng.choice(["interleaved", "half"]),
                kind=kind, factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.0]))
    if op == "step":
        hi = _log_int(rng, 64, 32767)
        return dict(op=op, S=_log_int(rng, 1, 700), page=rng.choice([16, 32, 64, 128, 256]), ctx_lo=0, ctx_hi=hi,
                    new_hi=_log_int(rng, 1, 512), p_chunk=rng.uniform(0, 0.5), p_done=rng.uniform(0, 0.1),
                    pad=rng.randint(0, 100), lens=rng.randint(1, 10 ** 6))
    if op == "rope":
        n = _log_int(rng, 1, 4096)
        return dict(op=op, seqs=rng.randint(1, max(1, min(8, 8192 // n))), n=n, H=Hkv * group, Hkv=Hkv,
                    dtype=rng.choice(["bf16", "f32"]), inverse=rng.random() < 0.5,
                    pos_hi=rng.choice([4096, 32768, 131072]), **rope)
    if op == "append":
        T = _log_int(rng, 1, 6001)
        page = rng.choice([16, 32, 64, 128, 256])
        return dict(op=op, T=T, pad=rng.randint(0, 200), H=Hkv * group, Hkv=Hkv, page=page,
                    pages=(T + page - 1) // page + rng.randint(1, 60), pos_hi=rng.choice([8192, 32768, 131072]),
                    **rope)
    base = dict(op=op, H=Hkv * group, Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128, 256]),
                causal=rng.random() < 0.85, pad=rng.choice([0, 0, rng.randint(1, 40)]), lens=rng.randint(1, 10 ** 6))
    how = rng.choice(["decode", "verify", "chunk", "mixed"])
    if how == "decode":
        hi = _log_int(rng, 16, 32768)
        return dict(base, S=_log_int(rng, 1, max(1, min(256, 600000 // hi))), new_lo=1, new_hi=1, kv_lo=1, kv_hi=hi)
    if how == "verify":
        hi = _log_int(rng, 16, 9001)
        return dict(base, S=_log_int(rng, 1, 32), new_lo=2, new_hi=rng.randint(2, 16), kv_lo=16, kv_hi=hi + 16)
    if how == "chunk":
        n = _log_int(rng, 17, 1024)
        return dict(base, new=str(n), kv=str(n + _log_int(rng, 1, 16000)))
    S = rng.randint(2, 12)
    new = [1 if rng.random() < 0.6 else _log_int(rng, 2, 300) for _ in range(S)]
    kv = [n + (0 if rng.random() < 0.3 else _log_int(rng, 1, 4000)) for n in new]
    return dict(base, new=" ".join(map(str, new)), kv=" ".join(map(str, kv)))


# ----------------------------------------------- what a case fixes: lengths --
def _step_lens(case):
    r = np.random.default_rng(case["lens"])
    S = case["S"]
    ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, S)
    new = np.ones(S, dtype=np.int64)
    chunk = r.random(S) < case["p_chunk"]
    new[chunk] = r.integers(1, case["new_hi"] + 1, int(chunk.sum()))
    done = r.random(S) < case["p_done"]
    new[done] = -1
    return ctx.astype(np.int64), new


def _extend_lens(case):
    if "new" in case:
        return np.array(case["new"].split(), dtype=np.int64), np.array(case["kv"].split(), dtype=np.int64)
    r = np.random.default_rng(case["lens"])
    new = r.integers(case["new_lo"], case["new_hi"] + 1, case["S"])
    kv = np.maximum(r.integers(case["kv_lo"], case["kv_hi"] + 1, case["S"]), new)
    return new.astype(np.int64), kv.astype(np.int64)


def _up(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "step":
        ctx, new = _step_lens(case)
        n = np.maximum(new, 0)
        T = int(n.sum()) + case["pad"]
        taken = np.where(new >= 0, _up(ctx + n, case["page"]) - _up(ctx, case["page"]), 0).sum()
        freed = np.where(new < 0, _up(ctx, case["page"]), 0).sum()
        # lengths in, offsets and lengths out, two entries a token out, a table entry a touched page in, new entries
        # out, ring entries in and out
        touched = np.where(n > 0, _up(ctx + n, case["page"]) - ctx // case["page"], 0).sum()
        return {"bytes": float(4 * (4 * len(ctx) + 2 * T + touched + 2 * taken + 2 * freed + 9)), "flops": 0.0}
    if op == "rope":
        T, e = case["seqs"] * case["n"], 2 if case["dtype"] == "bf16" else 4
        rows = case["H"] + case["Hkv"]
        return {"bytes": float(T * (rows * 2 * case["d"] * e * 2 + 4) + min(T, case["pos_hi"]) * case["rot"] * 4),
                "flops": float(T * rows * 2 * case["rot"] * 3)}
    if op == "append":
        T, e = case["T"], 2
        rows = case["H"] + 2 * case["Hkv"]
        return {"bytes": float(T * (rows * 2 * case["d"] * e * 2 + 8) + min(T, case["pos_hi"]) * case["rot"] * 4),
                "flops": float(T * (case["H"] + case["Hkv"]) * 2 * case["rot"] * 3)}
    new, kv = _extend_lens(case)
    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    if case["causal"]:
        pairs = sum(int(n) * int(L - n) + int(n) * (int(n) + 1) // 2 for n, L in zip(new, kv))
    else:
        pairs = int((new * kv).sum())
    bytes_ = int(kv.sum()) * Hkv * 8 * d + int(new.sum()) * H * 8 * d + 4 * int(_up(kv, case["page"]).sum())
    return {"bytes": float(bytes_), "flops": float(pairs * H * 12 * d)}


# ------------------------------------------------------------------- inputs --
def _randn(shape, g, dtype):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        b = min(flat.numel(), a + (1 << 28))
        flat[a:b] = torch.randn(b - a, generator=g, device=DEV, dtype=torch.float32).to(dtype)
    return out


def _angles(case):
    """Angle per position of each rotated pair, and the factor on cos and sin: the table's definition."""
    r, s, base = case["rot"], case["factor"], 10000.0
    j = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    if case["kind"] == "ntk":
        base = base * s ** (r / (r - 2))
    f = base ** (-2.0 * j / r)
    m = 1.0
    if case["kind"] == "linear":
        f = f / s
    elif case["kind"] == "yarn":
        turns = 4096 * f / (2 * math.pi)
        ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * ramp + f / s * (1.0 - ramp)
        m = 0.1 * math.log(s) + 1.0
    return f, m


def _table(case):
    if own:
        from differential_attention_04_b200 import api
        kind = {"none": api.ROPE_PLAIN, "linear": api.ROPE_LINEAR, "ntk": api.ROPE_NTK, "yarn": api.ROPE_YARN}
        return api.rope_table_scaled(case["pos_hi"], case["rot"], 10000.0, kind[case["kind"]], case["factor"],
                                     orig_len=4096, device=torch.device(DEV))
    f, m = _angles(case)
    a = torch.arange(case["pos_hi"], dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([a.cos() * m, a.sin() * m], -1).float()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = np.random.default_rng(seed + 17)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    st = {"case": case}
    op = case["op"]
    if op == "step":
        ctx, new = _step_lens(case)
        P = case["page"]
        held = _up(ctx, P)
        n = np.maximum(new, 0)
        taken = int(np.where(new >= 0, _up(ctx + n, P) - held, 0).sum())
        total = int(held.sum()) + taken + 50
        ids = r.permutation(total)
        width = int(_up(ctx + n, P).max()) + 2
        bt = np.full((len(ctx), width), -1, dtype=np.int64)
        at = 0
        for s, h in enumerate(held):
            bt[s, :h] = ids[at:at + h]
            at += h
        free = ids[at:]
        head = int(r.integers(0, total))
        ring = np.full(total, -1, dtype=np.int64)
        ring[(head + np.arange(len(free))) % total] = free
        st.update(ctx=i32(ctx), new=i32(new), bt=i32(bt), ring=i32(ring), pool=i32([head, len(free)]),
                  T=int(n.sum()) + case["pad"], page=P, pool_out=torch.zeros(2, dtype=torch.int32, device=DEV))
        return st
    if op == "rope":
        T = case["seqs"] * case["n"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        first = r.integers(0, case["pos_hi"] - case["n"] + 1, case["seqs"])
        pos = (first[:, None] + np.arange(case["n"])).reshape(-1)
        st.update(q=_randn((T, case["H"], 2, case["d"]), g, dt), k=_randn((T, case["Hkv"], 2, case["d"]), g, dt),
                  pos=i32(pos), table=_table(case))
        st.update(qo=torch.empty_like(st["q"]), ko=torch.empty_like(st["k"]))
        return st
    if op == "append":
        T, R, d, bf = case["T"], case["T"] + case["pad"], case["d"], torch.bfloat16
        rows = case["pages"] * case["page"]
        pos = np.concatenate([r.integers(0, case["pos_hi"], T), np.full(case["pad"], -1)])
        slots = np.concatenate([r.permutation(rows)[:T], np.full(case["pad"], -1)])
        st.update(q=_randn((R, case["H"], 2, d), g, bf), k=_randn((R, case["Hkv"], 2, d), g, bf),
                  v=_randn((R, case["Hkv"], 2 * d), g, bf), pos=i32(pos), slots=i32(slots), table=_table(case),
                  kc=_randn((case["pages"], case["page"], case["Hkv"], 2, d), g, bf),
                  vc=_randn((case["pages"], case["page"], case["Hkv"], 2 * d), g, bf))
        st["qo"] = torch.zeros_like(st["q"])
        return st
    new, kv = _extend_lens(case)
    H, Hkv, d, P = case["H"], case["Hkv"], case["d"], case["page"]
    T = int(new.sum()) + case["pad"]
    held = _up(kv, P)
    total = int(held.sum()) + 3
    ids = r.permutation(total)
    bt = np.full((len(kv), int(held.max()) + 1), -1, dtype=np.int64)
    at = 0
    for s, h in enumerate(held):
        bt[s, :h] = ids[at:at + h]
        at += h
    bf = torch.bfloat16
    st.update(q=_randn((T, H, 2, d), g, bf), kc=_randn((total, P, Hkv, 2, d), g, bf),
              vc=_randn((total, P, Hkv, 2 * d), g, bf), bt=i32(bt), new=new.tolist(), kv=kv.tolist(),
              cu=i32(np.concatenate([[0], np.cumsum(new)])), kvl=i32(kv), causal=case["causal"],
              lam=torch.rand(1, generator=g, device=DEV) * 0.8 + 0.1,
              w=1.0 + 0.02 * torch.randn(2 * d, generator=g, device=DEV),
              out=torch.zeros((T, H, 2 * d), dtype=bf, device=DEV))
    if own:
        # the schedule, made once a step and used by every layer, and the layers' shared workspace
        from differential_attention_04_b200 import api
        st["plan"] = api.extend_plan(st["cu"], st["kvl"], T, H, Hkv, d, int(new.max()), causal=case["causal"])
        st["ws"] = torch.empty(max(16, api.extend_workspace_size(st["plan"])), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- one pass --
def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def _run_own(st):
    from differential_attention_04_b200 import api
    case, op = st["case"], st["case"]["op"]
    if op == "step":
        cu, kv, pos, slots, info = api.paged_step(st["ctx"], st["new"], st["bt"], st["ring"], st["pool"], st["page"],
                                                  st["T"], pool_out=st["pool_out"])
        return st["bt"], st["ring"], st["pool_out"], cu, kv, pos, slots, info
    if op == "extend":
        return api.diffattn_extend(st["q"], st["kc"], st["vc"], st["bt"], st["plan"], st["lam"], LAMBDA_INIT, st["w"],
                                   EPS, workspace=st["ws"], out=st["out"])
    layout = api.ROPE_HALF if case["layout"] == "half" else api.ROPE_INTERLEAVED
    if op == "rope":
        return api.rope(st["q"], st["k"], st["pos"], st["table"], layout, inverse=case["inverse"],
                        out=(st["qo"], st["ko"]))
    q = api.kv_append(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["table"], st["kc"], st["vc"], layout,
                      out=st["qo"])
    return q, st["kc"], st["vc"]


def _plain_step(st):
    P, T, F = st["page"], st["T"], st["ring"].numel()
    ctx, new, bt, ring = st["ctx"].long(), st["new"].long(), st["bt"].long(), st["ring"].long()
    S, width = bt.shape
    head, count = st["pool"].long()
    done = new < 0
    n = new.clamp(min=0)
    old = (ctx + P - 1) // P
    want = torch.where(done, old, (ctx + n + P - 1) // P)
    need = want - old
    rel = torch.where(done, old, 0)
    tok_end, need_end, rel_end = n.cumsum(0), need.cumsum(0), rel.cumsum(0)
    total, taken, freed = tok_end[-1], need_end[-1], rel_end[-1]
    bad = (taken > count).long() + 2 * (want > width).any().long() + 4 * (total > T).long()
    ok = bad == 0
    col = torch.arange(width, device=DEV)
    mine = (col >= old[:, None]) & (col < want[:, None]) & ok
    src = (head + (need_end - need)[:, None] + col - old[:, None]) % F
    table = torch.where(mine, ring[src.clamp(min=0)], bt)
    give = (col < rel[:, None]) & ok
    dst = torch.where(give, (head + count + (rel_end - rel)[:, None] + col) % F, F)
    ring = torch.cat([ring, ring.new_zeros(1)]).scatter(0, dst.view(-1), bt.view(-1))[:F]
    cu = torch.cat([tok_end.new_zeros(1), tok_end]) * ok
    t = torch.arange(T, device=DEV)
    s = torch.searchsorted(tok_end, t, right=True).clamp(max=S - 1)
    live = (t < total) & ok
    pos = torch.where(live, ctx[s] + t - (tok_end - n)[s], -1)
    page = table[s, (pos // P).clamp(0, width - 1)]
    slots = torch.where(live, page * P + pos % P, -1)
    kv = torch.where(done, 0, ctx + n) * ok
    pool = torch.where(ok, torch.stack([(head + taken) % F, count - taken + freed]), torch.stack([head, count]))
    info = torch.stack([total, taken, freed, bad])
    return tuple(x.int() for x in (table, ring, pool, cu, kv, pos, slots, info))


def _rotate(x, table, pos, layout, inverse):
    """x [T, heads, 2, d] float32 with its first channels rotated at pos (rows of the table)."""
    cs = table[pos.clamp(min=0).long()][:, None, None]
    c, s = cs[..., 0], cs[..., 1]
    if inverse:
        s = -s
    half = c.shape[-1]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, a * s + b * c
    return y


def _plain_rope(st):
    case = st["case"]
    return tuple(_rotate(st[n].float(), st["table"], st["pos"], case["layout"], case["inverse"]).to(st[n].dtype)
                 for n in ("q", "k"))


def _plain_append(st):
    case = st["case"]
    T, bf = case["T"], torch.bfloat16
    rot = lambda x: _rotate(x[:T].float(), st["table"], st["pos"][:T], case["layout"], False).to(bf)
    st["qo"][:T] = rot(st["q"])
    rows = st["slots"][:T].long()
    st["kc"].view(-1, *st["kc"].shape[2:])[rows] = rot(st["k"])
    st["vc"].view(-1, *st["vc"].shape[2:])[rows] = st["v"][:T]
    return st["qo"], st["kc"], st["vc"]


def _plain_extend(st):
    case = st["case"]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    G, out, at = H // Hkv, st["out"].clone(), 0
    for s, (n, L) in enumerate(zip(st["new"], st["kv"])):
        pages = st["bt"][s, :_up(L, case["page"])].long()
        k = st["kc"][pages].view(-1, Hkv, 2, d)[:L].float().permute(1, 2, 3, 0)            # [Hkv, 2, d, L]
        v = st["vc"][pages].view(-1, Hkv, 2 * d)[:L].float().transpose(0, 1)                # [Hkv, L, 2d]
        q = st["q"][at:at + n].float().view(n, Hkv, G, 2, d).permute(1, 3, 2, 0, 4).reshape(Hkv, 2, G * n, d)
        x = torch.matmul(q, k) * (1.0 / math.sqrt(d))                                        # [Hkv, 2, G n, L]
        if st["causal"]:
            seen = torch.arange(L, device=DEV) <= torch.arange(L - n, L, device=DEV)[:, None]
            x = x.view(Hkv, 2, G, n, L).masked_fill(~seen, -math.inf).view(Hkv, 2, G * n, L)
        x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
        x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
        x = torch.matmul(x[:, 0] - st["lam"] * x[:, 1], v)                                   # [Hkv, G n, 2d]
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["w"] * (1.0 - LAMBDA_INIT)
        out[at:at + n] = y.view(Hkv, G, n, 2 * d).permute(2, 0, 1, 3).reshape(n, H, 2 * d).to(out.dtype)
        at += n
    return out


_PLAIN = {"step": _plain_step, "rope": _plain_rope, "append": _plain_append, "extend": _plain_extend}


# ------------------------------------------------- the definition, in 64 bits --
def _exact_rotate(x, pos, case, sign):
    """Each pair (a, b) as the complex number a + ib, times m exp(i sign n theta)."""
    r, d = case["rot"], case["d"]
    freq, m = _angles(case)
    turn = torch.polar(torch.full_like(freq, m).expand(len(pos), -1).contiguous(),
                       sign * pos.double()[:, None] * freq)[:, None, None]
    x = x.double()
    pairs = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half" \
        else x[..., :r].unflatten(-1, (r // 2, 2))
    z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
    if case["layout"] == "half":
        z = z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., r:]], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "step":
        return _exact_step(case, st)
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return tuple(_exact_rotate(st[n], st["pos"], case, sign) for n in ("q", "k"))
    if op == "append":
        T = case["T"]
        q, kc, vc = st["qo"].double(), st["kc"].double(), st["vc"].double()
        page, off = st["slots"][:T].long() // case["page"], st["slots"][:T].long() % case["page"]
        q[:T] = _exact_rotate(st["q"][:T], st["pos"][:T], case, 1.0)
        kc[page, off] = _exact_rotate(st["k"][:T], st["pos"][:T], case, 1.0)
        vc[page, off] = st["v"][:T].double()
        return q, kc, vc
    return _exact_extend(case, st)


def _exact_step(case, st):
    """Request by request, as a scheduler on the host would."""
    ctx, new = _step_lens(case)
    P, T = case["page"], st["T"]
    bt, ring = st["bt"].cpu().numpy().copy(), st["ring"].cpu().numpy().copy()
    head, count = (int(x) for x in st["pool"])
    F, cu, kv, pos, slots = len(ring), [0], [], [], []
    take, back = head, head + count
    taken = freed = 0
    for s in range(len(ctx)):
        c, n = int(ctx[s]), int(new[s])
        if n < 0:
            for j in range(_up(c, P)):
                ring[back % F] = bt[s, j]
                back, freed = back + 1, freed + 1
            cu.append(cu[-1])
            kv.append(0)
            continue
        for j in range(_up(c, P), _up(c + n, P)):
            bt[s, j] = ring[take % F]
            take, taken = take + 1, taken + 1
        for p in range(c, c + n):
            pos.append(p)
            slots.append(int(bt[s, p // P]) * P + p % P)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pos += [-1] * (T - len(pos))
    slots += [-1] * (T - len(slots))
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    return tuple(i32(x) for x in (bt, ring, [take % F, count - taken + freed], cu, kv, pos, slots,
                                  [cu[-1], taken, freed, 0]))


def _exact_extend(case, st):
    """Head by head and map by map, through log-sum-exp."""
    H, G, d, P = case["H"], case["H"] // case["Hkv"], case["d"], case["page"]
    out, lam, w, start = st["out"].double(), st["lam"].double(), st["w"].double(), 0
    for s, (n, L) in enumerate(zip(st["new"], st["kv"])):
        where = torch.arange(L, device=DEV)
        page, off = st["bt"][s].long()[where // P], where % P
        last = torch.arange(n, device=DEV)[:, None] + (L - n) if case["causal"] else L
        hidden = where[None, :] > last if case["causal"] else None
        for h in range(H):
            kh, vh = st["kc"][page, off, h // G].double(), st["vc"][page, off, h // G].double()
            o = 0
            for i in range(2):
                lg = st["q"][start:start + n, h, i].double() @ kh[:, i].T / d ** 0.5
                if hidden is not None:
                    lg = lg.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(lg, -1, keepdim=True)
                a = torch.exp(lg - torch.where(z == -math.inf, torch.zeros_like(z), z)) @ vh
                o = a if i == 0 else o - lam * a
            rms = (o * o).sum(-1, keepdim=True) / (2 * d)
            out[start:start + n, h] = (1 - LAMBDA_INIT) * w * o / (rms + EPS).sqrt()
        start += n
    return out
