"""The attention side of a block-decoding layer, as measured work: the paged key-value cache
(written, quantised as it is written, and read back), attention of a few new tokens over it, and
the gated residual with the norms before and after a block.

``own = False`` runs each operator in its plain form (elementary torch operations in 32 bits);
``own = True`` makes the calls a user makes of ``moe_expert_step_gb300``.  Both take the same
state.  Every case is a dict with an operator's name in ``op``:

* ``write``  kv_cache_write: [R*n][Hkv][D] keys and values (rows of a fused projection, so the
  token stride is larger than Hkv*D) go to the pages that hold positions pos[R][n]; a negative
  position writes nothing.  FP8 caches hold E4M3 codes and one power-of-two exponent for each
  token and head: the smallest e with max|x| <= 448 * 2^e, biased by 127 in one byte.
* ``read``   kv_cache_read: the values at positions pos[R][n], dense (zeros where negative).
* ``attend`` block_attention: n_q new tokens of each request over the first kv_len[r] positions,
  the last n_q of which are the new tokens themselves; in-block bidirectional, or causal, and
  optionally within a window.
* ``norm``   block_residual_norm: h' = h + s * gate * w_post * y / rms(y), x = w_pre * h' / rms(h').
"""
import math

import torch

own = False

V_MODEL = dict(E=256, k=8, I=512, Is=512, V=152064)  # the block step's own layer, around the norm

# ------------------------------------------------------------------------------------- cases


def _attend(name, dtype, R, n_q, length, Hq, Hkv, D, page, causal=False, window=0, ragged=False, lse=False):
    return dict(name=name, op="attend", dtype=dtype, R=R, n_q=n_q, length=length, Hq=Hq, Hkv=Hkv, D=D, page=page,
                causal=causal, window=window, ragged=ragged, lse=lse)


def _copy(name, op, dtype, R, n, length, Hkv, D, page):
    return dict(name=name, op=op, dtype=dtype, R=R, n=n, length=length, Hkv=Hkv, D=D, page=page)


def _norm(name, T, H, P, y_dtype, dtype="bf16", post=True, gate=True):
    return dict(name=name, op="norm", dtype=dtype, T=T, H=H, P=P, y_dtype=y_dtype, post=post, gate=gate)


def listed():
    return [
        # one user's next token early in a conversation: latency alone counts
        _attend("attend_token_short", "bf16", 1, 1, 203, 16, 2, 128, 16),
        # next tokens of sixteen users with conversations of very different lengths, one slot idle
        _attend("attend_token_ragged", "bf16", 16, 1, 8192, 16, 2, 128, 64, causal=True, ragged=True),
        # one token over a very long document in a quantised cache; the statistics are kept, for
        # joining with attention over another cache
        _attend("attend_token_long_fp8", "fp8", 1, 1, 131072, 16, 2, 128, 64, lse=True),
        # a masked block of 32 tokens of one request, bidirectional in the block, over its prefix
        _attend("attend_block", "bf16", 1, 32, 16384, 16, 2, 128, 64),
        # the same for a batch of sixteen requests over long prefixes in a quantised cache
        _attend("attend_block_batch_fp8", "fp8", 16, 32, 32768, 16, 2, 128, 64, ragged=True),
        # a short odd block with narrow heads, causal and within a sliding window, full precision
        _attend("attend_window_f32", "f32", 3, 7, 1001, 8, 4, 64, 16, causal=True, window=500, lse=True),
        # a decoding round's block enters the cache
        _copy("write_block", "write", "bf16", 1, 32, 16384, 2, 128, 64),
        # prompts enter a quantised cache
        _copy("write_prompt_fp8", "write", "fp8", 8, 4096, 4096, 8, 128, 64),
        # the last odd stretch of a prefix is read back, to be handed over or checked
        _copy("read_prefix", "read", "bf16", 1, 777, 4001, 2, 64, 16),
        # whole prefixes are read back from a quantised cache
        _copy("read_prompt_fp8", "read", "fp8", 8, 4096, 4096, 8, 128, 64),
        # after the experts of one 32-token block (their output is fp32)
        _norm("norm_block", 32, 2048, 32, "f32"),
        # after the attention of a large batch (its projected output is bf16)
        _norm("norm_batch", 8192, 2048, 32, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read", "norm"])
    if op == "norm":
        P = rng.choice([1, 8, 32, 64])
        T = _log(rng, 1, 8192)
        H = 128 * rng.choice([2, 4, 5, 8, 11, 16, 20, 32, 40])
        T = max(1, min(_odd(T), 4900 * 2048 // H))
        c = _norm("", T, H, P, rng.choice(["f32", "bf16"]), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.8,
                  rng.random() < 0.8)
        del c["name"]
        return c
    dtype = rng.choice(["bf16", "bf16", "fp8", "fp8", "f32"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op != "attend":
        n = _log(rng, 1, 4096)
        R = _log(rng, 1, 16)
        while R * n * Hkv * D * {"f32": 16, "bf16": 8, "fp8": 6}[dtype] > 2e8:
            R, n = max(1, R // 2), max(1, n // 2)
        n = _odd(n)
        c = _copy("", op, dtype, R, n, _odd(n + _log(rng, 1, 4096)), Hkv, D, page)
    else:
        G = rng.choice([1, 2, 4, 8, 16])
        if dtype == "f32":  # the accuracy path: small models
            R, n_q, length = _log(rng, 1, 8), _log(rng, 1, 8), _log(rng, 8, 2048)
        else:
            R, n_q, length = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 8, 16, 32, 32, 64]), _log(rng, 8, 131072)
        length = max(length, n_q)
        size = {"f32": 4, "bf16": 2, "fp8": 1}[dtype]
        while (R * length * n_q * G * Hkv * D > 16 * 32 * 32768 * 16 * 128 // 2
               or 2 * R * Hkv * D * (length * size + n_q * G * max(size, 2)) > 1.4e8):
            R, length = max(1, R // 2), max(n_q, length // 2)
        c = _attend("", dtype, R, n_q, _odd(max(length, n_q)), G * Hkv, Hkv, D, page, rng.random() < 0.4,
                    rng.choice([0, 0, 0, _odd(_log(rng, 16, 4096))]), rng.random() < 0.7, rng.random() < 0.4)
    del c["name"]
    return c


def _odd(n):
    """n, or the odd number above it where it is a multiple of 1024."""
    return n + 1 if n % 1024 == 0 else n


def _lengths(c):
    """Cached positions of each request: the longest first; in a ragged batch the others spread
    down to a quarter of it, and of four or more one is an idle slot."""
    if not c["ragged"]:
        return [c["length"]] * c["R"]
    n = [max(min(c["n_q"], c["length"]), c["length"] - (3 * c["length"] * ((7 * r) % c["R"])) // (4 * c["R"]))
         for r in range(c["R"])]
    if c["R"] >= 4:
        n[c["R"] // 2] = 0
    return n


# ------------------------------------------------------------------------------------- inputs

ACT = {"bf16": torch.bfloat16, "fp8": torch.bfloat16, "f32": torch.float32}
STORE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "f32": torch.float32}


def _quantise(x):
    """E4M3 values and biased exponents of x [..., D]: e is the smallest with max|x| <= 448 * 2^e,
    kept within [-100, 119]; infinities saturate, NaN stays NaN."""
    x = x.float()
    amax = torch.nan_to_num(x.abs(), nan=0.0).amax(-1).clamp(max=torch.finfo(torch.float32).max)
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 119)
    q = (x * torch.exp2(-e.float()).unsqueeze(-1)).clamp(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _dequantise(q, e):
    return q.float() * torch.exp2(e.float() - 127.0).unsqueeze(-1)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _heads(shape, g, dtype):
    """Key or value vectors: normal, with a strength of their own for each token and head."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(0.4 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))).to(dtype)


def _pool(c, lengths, g):
    """A cache whose pages are in no order and hold old values wherever nothing was written."""
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    need = [-(-n // page) for n in lengths]
    max_pages = max(max(need), 1)
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.full((c["R"], max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    s = dict(table=table, n_pages=n_pages, max_pages=max_pages)
    for name in ("k", "v"):
        x = _heads((n_pages, Hkv, page, D), g, torch.bfloat16 if c["dtype"] == "fp8" else ACT[c["dtype"]])
        if c["dtype"] == "fp8":
            s[name], s[name + "_exp"] = _quantise(x)
        else:
            s[name], s[name + "_exp"] = x, None
        del x
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "norm":
        T, H, P = c["T"], c["H"], c["P"]
        s["y"] = (0.3 * torch.randn((T, H), generator=g, device="cuda")).to(ACT[c["y_dtype"]])
        s["h"] = 2.0 * torch.randn((T, H), generator=g, device="cuda")
        s["gate"] = 0.5 + 0.5 * torch.randn((-(-T // P), H), generator=g, device="cuda") if c["gate"] else None
        w = lambda: (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(ACT[c["dtype"]])  # noqa: E731
        s["w_post"], s["w_pre"] = w() if c["post"] else None, w()
        s["h_out"] = torch.empty_like(s["h"])
        s["x"] = torch.empty((T, H), dtype=ACT[c["dtype"]], device="cuda")
    elif c["op"] == "attend":
        lengths = _lengths(c)
        s |= _pool(c, lengths, g)
        s["kv_len"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        T, Hq, D = c["R"] * c["n_q"], c["Hq"], c["D"]
        s["q"] = (1.5 * torch.randn((T, Hq, D), generator=g, device="cuda")).to(ACT[c["dtype"]])
        s["out"] = torch.empty((T, Hq, D), dtype=ACT[c["dtype"]], device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda") if c["lse"] else None
        s["scale"] = D ** -0.5
    else:
        s |= _pool(c, [c["length"]] * c["R"], g)
        T, n, Hkv, D = c["R"] * c["n"], c["n"], c["Hkv"], c["D"]
        first = c["length"] - n  # the last n positions of each request
        pos = torch.arange(first, first + n, device="cuda", dtype=torch.int32).repeat(c["R"], 1)
        if c["op"] == "read" and n >= 8:
            pos[-1, n // 2] = -1  # a padding token
        s["pos"] = pos.contiguous()
        if c["op"] == "write":  # keys and values are parts of one projected row of each token
            s["kv"] = _heads((T, 2 * Hkv, D), g, ACT[c["dtype"]])
        else:
            s["k_out"] = torch.empty((T, Hkv, D), dtype=ACT[c["dtype"]], device="cuda")
            s["v_out"] = torch.empty_like(s["k_out"])
    if own:  # the handles and the workspace that a program keeps
        import moe_expert_step_gb300 as ms
        kind = {"bf16": ms.BF16, "f32": ms.F32, "fp8": ms.FP8}
        if c["op"] == "norm":
            s["dims"] = ms.ModelDims(H=c["H"], P=c["P"], dtype=kind[c["dtype"]], **V_MODEL)
        else:
            s["dims"] = ms.KvDims(Hq=c.get("Hq", c["Hkv"]), Hkv=c["Hkv"], D=c["D"], page=c["page"],
                                  n_pages=s["n_pages"], max_pages=s["max_pages"], dtype=kind[c["dtype"]])
            s["cache"] = ms.kv_cache(s["k"], s["v"], s["table"], s["k_exp"], s["v_exp"])
            s["ws"] = ms.kv_workspace(s["dims"], c["R"], c.get("n_q", 1))
    return s


# ------------------------------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"norm": _plain_norm, "attend": _plain_attend, "write": _plain_write, "read": _plain_read}[c["op"]](s, c)


def _cache_out(s):
    out = dict(k=s["k"], v=s["v"])
    if s["k_exp"] is not None:
        out |= dict(k_exp=s["k_exp"], v_exp=s["v_exp"])
    return out


def _run_own(s, c):
    import moe_expert_step_gb300 as ms
    if c["op"] == "norm":
        ms.block_residual_norm(s["dims"], s["y"], s["h"], s["h_out"], s["x"], w_pre=s["w_pre"], w_post=s["w_post"],
                               gate=s["gate"], res_scale=0.7, eps=1e-6)
        return dict(h=s["h_out"], x=s["x"])
    if c["op"] == "write":
        Hkv = c["Hkv"]
        ms.kv_cache_write(s["dims"], c["R"], s["kv"][:, :Hkv], s["kv"][:, Hkv:], s["pos"], s["cache"], s["ws"])
        return _cache_out(s)
    if c["op"] == "read":
        ms.kv_cache_read(s["dims"], c["R"], s["pos"], s["cache"], s["k_out"], s["v_out"], s["ws"])
        return dict(k=s["k_out"], v=s["v_out"])
    ms.block_attention(s["dims"], c["R"], s["q"], s["kv_len"], s["cache"], s["out"], s["ws"], s["scale"],
                       causal=c["causal"], window=c["window"], lse=s["lse"])
    return dict(out=s["out"]) if s["lse"] is None else dict(out=s["out"], lse=s["lse"])


def _plain_norm(s, c):
    y = s["y"].float()
    if s["w_post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].repeat_interleave(c["P"], 0)[:c["T"]]
    h = s["h"] + 0.7 * y
    x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w_pre"].float()
    return dict(h=h, x=x.to(s["x"].dtype))


def _places(s, c):
    """Page and place in the page of every position that is not negative, and which those are."""
    live = s["pos"] >= 0
    pos = s["pos"].long().clamp(min=0)
    pages = torch.gather(s["table"].long(), 1, pos // c["page"])
    return pages.reshape(-1), (pos % c["page"]).reshape(-1), live.reshape(-1)


def _plain_write(s, c):
    pages, at, _ = _places(s, c)  # every measured token is written
    for name, x in (("k", s["kv"][:, :c["Hkv"]]), ("v", s["kv"][:, c["Hkv"]:])):
        if c["dtype"] == "fp8":
            q, e = _quantise(x)
            s[name].view(torch.uint8)[pages, :, at] = q.view(torch.uint8)
            s[name + "_exp"][pages, :, at] = e
        else:
            s[name][pages, :, at] = x
    return _cache_out(s)


def _plain_read(s, c):
    pages, at, live = _places(s, c)
    out = {}
    for name in ("k", "v"):
        pages_l, at_l = torch.where(live, pages, 0), torch.where(live, at, 0)
        x = s[name].view(torch.uint8)[pages_l, :, at_l].view(s[name].dtype) if c["dtype"] == "fp8" else s[name][pages_l, :, at_l]
        x = _dequantise(x, s[name + "_exp"][pages_l, :, at_l]) if c["dtype"] == "fp8" else x.float()
        out[name] = torch.where(live[:, None, None], x, 0.0).to(ACT[c["dtype"]])
    return out


def _plain_attend(s, c):
    R, n_q, Hq, Hkv, D = c["R"], c["n_q"], c["Hq"], c["Hkv"], c["D"]
    G, N = Hq // Hkv, s["max_pages"] * c["page"]
    pages = s["table"].long().clamp(min=0)
    kv = []
    for name in ("k", "v"):
        x = s[name].view(torch.uint8)[pages].view(s[name].dtype) if c["dtype"] == "fp8" else s[name][pages]
        x = _dequantise(x, s[name + "_exp"][pages]) if c["dtype"] == "fp8" else x.float()
        kv.append(x.transpose(1, 2).reshape(R, Hkv, N, D))
    q = s["q"].float().view(R, n_q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n_q * G, D)
    score = (q @ kv[0].transpose(-1, -2)).view(R, Hkv, n_q, G, N) * s["scale"]
    j = torch.arange(N, device="cuda")
    length = s["kv_len"].long()[:, None, None]
    at = length - n_q + torch.arange(n_q, device="cuda")[None, :, None]
    see = (j < length).expand(R, n_q, N)
    if c["causal"]:
        see = see & (j <= at)
    if c["window"]:
        see = see & (j > at - c["window"])
    score = score.masked_fill(~see[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where((j < length)[:, None, 0, :, None], kv[1], 0.0)
    out = (p.view(R, Hkv, n_q * G, N) @ v).view(R, Hkv, n_q, G, D) / torch.where(total > 0, total, 1.0)
    out = out.permute(0, 2, 1, 3, 4).reshape(R * n_q, Hq, D).to(s["out"].dtype)
    if s["lse"] is None:
        return dict(out=out)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(R * n_q, Hq)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------------------------- definitions


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, request by request."""
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "norm":
        y, h = s["y"].to(f64), s["h"].to(f64)
        if s["w_post"] is not None:
            y = s["w_post"].to(f64) * y / torch.sqrt((y * y).sum(1, keepdim=True) / c["H"] + 1e-6)
        if s["gate"] is not None:
            y = y * s["gate"].to(f64)[torch.arange(c["T"], device="cuda") // c["P"]]
        h = h + 0.7 * y
        return dict(h=h, x=s["w_pre"].to(f64) * h / torch.sqrt((h * h).sum(1, keepdim=True) / c["H"] + 1e-6))

    def stored(name):  # [n_pages][Hkv][page][D]
        x = s[name].to(torch.float32).to(f64)
        return x if s[name + "_exp"] is None else torch.ldexp(x, s[name + "_exp"].to(torch.int32).unsqueeze(-1) - 127)

    page = c["page"]
    if c["op"] == "write":
        out, Hkv = {}, c["Hkv"]
        for name, x in (("k", s["kv"][:, :Hkv]), ("v", s["kv"][:, Hkv:])):
            new = x.to(f64).reshape(c["R"], c["n"], Hkv, c["D"])
            pool = s[name].to(torch.float32).to(f64)
            exps = s[name + "_exp"]
            for r in range(c["R"]):
                keep = torch.nonzero(s["pos"][r] >= 0).flatten()
                p = s["pos"][r][keep].long()
                pages, val = s["table"][r].long()[p // page], new[r][keep]
                if exps is not None:
                    most = val.abs().amax(-1)
                    e = torch.ceil(torch.log2(most / 448.0)).clamp(-100, 119)
                    e = torch.where(most > 0, e, -100.0)
                    exps[pages, :, p % page] = (e + 127).to(torch.uint8)
                    val = val / torch.exp2(e).unsqueeze(-1)
                pool[pages, :, p % page] = val
            out[name] = pool
            if exps is not None:
                out[name + "_exp"] = exps
        return out
    if c["op"] == "read":
        out = {}
        for name in ("k", "v"):
            pool, rows = stored(name), []
            for r in range(c["R"]):
                p = s["pos"][r].long()
                x = pool[s["table"][r].long()[p.clamp(min=0) // page], :, p.clamp(min=0) % page]
                rows.append(x * (p >= 0)[:, None, None])
            out[name] = torch.cat(rows)
        return out
    n_q, Hq, Hkv, D = c["n_q"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    q = s["q"].to(f64)
    out = torch.zeros((c["R"] * n_q, Hq, D), dtype=f64, device="cuda")
    lse = torch.full((c["R"] * n_q, Hq), -math.inf, dtype=f64, device="cuda")
    for r, L in enumerate(_lengths(c)):
        if L == 0:
            continue
        ids = s["table"][r, :-(-L // page)].long()
        i = torch.arange(L, device="cuda")
        at = torch.arange(L - n_q, L, device="cuda")[:, None]
        hidden = (i > at) if c["causal"] else torch.zeros((n_q, L), dtype=torch.bool, device="cuda")
        if c["window"]:
            hidden = hidden | (i <= at - c["window"])
        for h in range(Hkv):
            kv = []
            for name in ("k", "v"):
                x = s[name][ids, h].to(torch.float32).to(f64)
                if s[name + "_exp"] is not None:
                    x = torch.ldexp(x, s[name + "_exp"][ids, h].to(torch.int32).unsqueeze(-1) - 127)
                kv.append(x.reshape(-1, D)[:L])
            rows = q[r * n_q:(r + 1) * n_q, h * G:(h + 1) * G]
            z = torch.einsum("igd,jd->igj", rows, kv[0]) * s["scale"]
            z = z.masked_fill(hidden[:, None, :], -math.inf)
            total = torch.logsumexp(z, -1)
            p = torch.nan_to_num(torch.exp(z - total[..., None]), nan=0.0)
            out[r * n_q:(r + 1) * n_q, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", p, kv[1])
            lse[r * n_q:(r + 1) * n_q, h * G:(h + 1) * G] = total
    return dict(out=out, lse=lse) if c["lse"] else dict(out=out)


# ------------------------------------------------------------------------------------- work


def work(case):
    """Bytes: inputs read once, outputs written once.  Flops: multiplications and additions of the
    visible query-key pairs (a cache's copies are counted as one operation a value)."""
    c = case
    act = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "norm":
        y = 4 if c["y_dtype"] == "f32" else 2
        n = c["T"] * c["H"]
        vec = c["H"] * act * (1 + c["post"]) + (4 * c["H"] * -(-c["T"] // c["P"]) if c["gate"] else 0)
        return dict(bytes=n * (y + 4 + 4 + act) + vec, flops=10 * n)
    token = c["Hkv"] * ((c["D"] + 1) if c["dtype"] == "fp8" else c["D"] * act)  # one token's keys, as cached
    if c["op"] in ("write", "read"):
        n = c["R"] * c["n"] - (c["op"] == "read" and c["n"] >= 8)
        return dict(bytes=2 * n * (token + c["Hkv"] * c["D"] * act) + 4 * c["R"] * c["n"],
                    flops=2 * n * c["Hkv"] * c["D"])
    seen = pairs = 0
    n_q, w = c["n_q"], c["window"]
    for L in _lengths(c):
        if L == 0:
            continue
        seen += L - (max(0, L - n_q - w + 1) if w else 0)
        for i in range(n_q):
            at = L - n_q + i
            hi = at + 1 if c["causal"] else L
            lo = max(0, at - w + 1) if w else 0
            pairs += max(0, hi - lo)
    qo = 2 * c["R"] * n_q * c["Hq"] * c["D"] * act
    return dict(bytes=qo + 2 * seen * token + (4 * c["R"] * n_q * c["Hq"] if c["lse"] else 0),
                flops=4 * c["D"] * c["Hq"] * pairs)
