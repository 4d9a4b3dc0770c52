"""What stands around the paged cache and beside attention in a decoder layer, as measured work:
pages and positions given out on the GPU, rotary positions of queries and keys, and the gated
delta rule, the token mixer whose history is a matrix a head.

``own = False`` runs each operator in its plain form (elementary torch operations in 32 bits);
``own = True`` makes the calls a user makes of ``moe_expert_step_gb300``.  Both take the same
state.  Every case is a dict with an operator's name in ``op``:

* ``plan``   kv_cache_plan: requests grow by n_new tokens (or drop their last -n_new): pages are taken
  from the front of a ring of free pages, or go back to its end, the page tables are extended,
  and every new token gets its position and its slot in the pool.
* ``rotary`` block_rotary: the first `rot` of the D elements of every query and key head are
  turned by pos * freq_i, in pairs (i, i + rot/2) or (2i, 2i+1), and multiplied by `mscale`; the
  others pass.  The frequencies may be scaled for contexts longer than the original one.
* ``delta``  block_delta_rule: for each token S <- e^g S + beta k (v - e^g S^T k)^T, o = scale * S^T q,
  with queries and keys normalised to length 1 first; states are kept a slot a request, transposed.
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------------- cases


def _plan(name, R, n, length, page, tight=False):
    return dict(name=name, op="plan", R=R, n=n, length=length, page=page, tight=tight)


def _rotary(name, dtype, R, n, length, Hq, Hkv, D, rot, interleaved=False, scaling="none", base=1e6):
    return dict(name=name, op="rotary", dtype=dtype, R=R, n=n, length=length, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                interleaved=interleaved, scaling=scaling, base=base)


def _delta(name, dtype, R, n, Hk, Hv, Dk, Dv, ragged=False, fresh=False, write=True):
    return dict(name=name, op="delta", dtype=dtype, R=R, n=n, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, ragged=ragged, fresh=fresh,
                write=write)


def listed():
    return [
        # a decoding round begins: one request's next block of 32 positions; latency alone counts
        _plan("plan_block", 1, 32, 16384, 64),
        # prompts of very different lengths arrive together, others end and give their pages back,
        # and there are too few pages for the last ones
        _plan("plan_prompts", 256, 4096, 8192, 16, tight=True),
        # queries and keys of one block, a quarter of the head rotated, far into a context
        _rotary("rotary_block", "bf16", 1, 32, 100000, 16, 2, 128, 32),
        # the same of long prompts, whole heads, frequencies ramped for a longer context
        _rotary("rotary_prompt", "bf16", 8, 4096, 8192, 16, 2, 128, 128, scaling="dimensions"),
        # an odd block with narrow heads in full precision, neighbouring elements paired
        _rotary("rotary_pairs_f32", "f32", 3, 1001, 20011, 8, 4, 64, 48, interleaved=True, scaling="rotations"),
        # one user's next token: latency alone counts
        _delta("delta_token", "bf16", 1, 1, 16, 32, 128, 128),
        # next tokens of many users: their states are read and written once
        _delta("delta_token_batch", "bf16", 128, 1, 16, 32, 128, 128),
        # a denoising round over a masked block: the history is read, and not yet changed
        _delta("delta_block", "bf16", 1, 32, 16, 32, 128, 128, write=False),
        # resolved blocks of a batch of requests, some of them shorter, enter their histories
        _delta("delta_block_batch", "bf16", 16, 32, 16, 32, 128, 128, ragged=True),
        # one user's long prompt, from nothing
        _delta("delta_prompt", "bf16", 1, 8192, 16, 32, 128, 128, fresh=True),
        # prompts of a batch, ragged, continuing earlier turns
        _delta("delta_prompt_batch", "bf16", 8, 4096, 16, 32, 128, 128, ragged=True),
        # a short odd stretch with narrow heads in full precision
        _delta("delta_stretch_f32", "f32", 3, 77, 2, 4, 64, 64, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rotary", "rotary", "delta", "delta", "delta", "delta"])
    if op == "plan":
        R, n = _log(rng, 1, 512), _log(rng, 1, 8192)
        while R * n > 1 << 20:
            R, n = max(1, R // 2), max(1, n // 2)
        c = _plan("", R, _odd(n), _odd(_log(rng, 16, 32768)), rng.choice([16, 32, 64, 128]), rng.random() < 0.3)
    elif op == "rotary":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        R, n = _log(rng, 1, 64), _log(rng, 1, 8192)
        while R * n * (Hq + Hkv) * D * (2 if dtype == "f32" else 1) > 8 * 4096 * 18 * 128:
            R, n = max(1, R // 2), max(1, n // 2)
        rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
        c = _rotary("", dtype, R, _odd(n), _odd(n + _log(rng, 1, 1000000)), Hq, Hkv, D, rot, rng.random() < 0.4,
                    rng.choice(["none", "linear", "rotations", "dimensions"]), rng.choice([1e4, 5e5, 1e6, 1e7]))
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
        Hk, Dk, Dv = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        Hv = Hk * rng.choice([1, 2, 2, 4])
        if dtype == "f32":  # the accuracy path: small models
            R, n, Hk = _log(rng, 1, 8), _log(rng, 1, 512), min(Hk, 4)
            Hv = min(Hv, 2 * Hk)
        else:
            R, n = _log(rng, 1, 128), rng.choice([1, 1, 2, 3, 5, 8, 16, 32, 32, 64] + [_log(rng, 65, 8192)] * 5)
        while R > 1 and (R * Hv * Dk * Dv > 128 * 32 * 128 * 128 or R * n * Hv * max(Dk, Dv) > 8 * 4096 * 32 * 128):
            R //= 2
        c = _delta("", dtype, R, _odd(n), Hk, Hv, Dk, Dv, rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.7)
    del c["name"]
    return c


def _odd(n):
    """n, or the odd number above it where it is a multiple of 1024."""
    return n + 1 if n % 1024 == 0 else n


# ------------------------------------------------------------------------------------- inputs

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
ORIGINAL, FACTOR = 4096, 8.0  # a context of 32768 where 4096 was the original one
RAMP = dict(rotations=(1.0, 4.0), dimensions=(1.0, 32.0), linear=(0.0, 0.0), none=(0.0, 0.0))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lengths(c):
    """Tokens of each request: all of them, or spread down to a quarter, and of four or more one idle."""
    R, n = c["R"], c["n"]
    if not c["ragged"]:
        return [n] * R
    out = [max(1, n - (3 * n * ((5 * r) % R)) // (4 * R)) for r in range(R)]
    if R >= 4:
        out[R // 2] = 0
    return out


def _mscale(c):
    return 0.1 * math.log(FACTOR) + 1.0 if c["scaling"] == "dimensions" else 1.0


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    i32 = lambda x: torch.as_tensor(x, device="cuda").to(torch.int32)  # noqa: E731
    if c["op"] == "plan":
        R, n, page = c["R"], c["n"], c["page"]
        rand = lambda lo, hi, k: torch.randint(lo, hi, (k,), generator=g, device="cuda")  # noqa: E731
        kv_len = rand(0, c["length"] + 1, R)
        m = rand(1, n + 1, R) if R > 1 else torch.full((1,), n, device="cuda")
        kind = rand(0, 8, R) if R > 1 else torch.ones(1, device="cuda")
        m = torch.where(kind == 0, -kv_len, m)  # an ended request
        m = torch.where(kind == 7, -torch.minimum(kv_len, rand(0, n + 1, R)), m)  # one cut back
        held = -(-kv_len // page)
        grow = (-(-(kv_len + m) // page) - held).clamp(min=0)
        max_pages = -(-(c["length"] + n) // page)
        n_pages = R * max_pages + 5
        free = int(grow.sum()) // 2 + 1 if c["tight"] else n_pages - int(held.sum())
        order = torch.randperm(n_pages, generator=g, device="cuda")
        i = torch.arange(max_pages, device="cuda")
        at = (held.cumsum(0) - held)[:, None] + i
        table = torch.where(i < held[:, None], order[at.clamp(max=n_pages - 1)], -1)
        first = int(rand(0, n_pages, 1))
        ring = torch.full((n_pages,), -1, device="cuda")
        ring[(first + torch.arange(free, device="cuda")) % n_pages] = order[n_pages - free:]
        s |= dict(kv_len=i32(kv_len), n_new=i32(m), table=i32(table), ring=i32(ring), head=i32([first, free]),
                  head_out=i32([0, 0]), n_pages=n_pages, max_pages=max_pages)
        s |= dict(new_len=i32([0] * R), pos=i32(torch.zeros((R, n))), slots=i32(torch.zeros((R, n))))
    elif c["op"] == "rotary":
        R, n, Hq, Hkv, D = c["R"], c["n"], c["Hq"], c["Hkv"], c["D"]
        T = R * n
        start = torch.randint(0, c["length"] - n + 1, (R, 1), generator=g, device="cuda")
        pos = start + torch.arange(n, device="cuda")
        if n >= 8:
            pos[-1, n - n // 8:] = -1  # padding behind a shorter request
        s["pos"] = i32(pos)
        row = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(ACT[c["dtype"]])
        s["qkv"] = row * torch.exp(0.4 * torch.randn((T, Hq + 2 * Hkv, 1), generator=g, device="cuda")).to(row.dtype)
        s["q_out"] = torch.zeros((T, Hq, D), dtype=ACT[c["dtype"]], device="cuda")
        s["k_out"] = torch.zeros((T, Hkv, D), dtype=ACT[c["dtype"]], device="cuda")
        s["freq"] = _frequencies(c)
    else:
        R, n, Hk, Hv, Dk, Dv = c["R"], c["n"], c["Hk"], c["Hv"], c["Dk"], c["Dv"]
        T, act = R * n, ACT[c["dtype"]]
        width = 2 * Hk * Dk + Hv * Dv
        # queries, keys and values are parts of one projected row, after an activation: their
        # elements have means of their own, so that neighbouring keys are alike
        x = torch.randn((T, width), generator=g, device="cuda")
        x = torch.nn.functional.silu(x + 0.5 * torch.randn(width, generator=g, device="cuda")).to(act)
        s["qkv"] = x
        s["q"] = x[:, :Hk * Dk].unflatten(1, (Hk, Dk))
        s["k"] = x[:, Hk * Dk:2 * Hk * Dk].unflatten(1, (Hk, Dk))
        s["v"] = x[:, 2 * Hk * Dk:].unflatten(1, (Hv, Dv))
        # each head forgets at a rate of its own, from a few tokens to thousands
        rate = torch.exp(torch.empty(Hv, device="cuda").uniform_(math.log(1e-4), math.log(2.0), generator=g))
        s["g"] = -rate * torch.exp(0.5 * torch.randn((T, Hv), generator=g, device="cuda"))
        s["beta"] = torch.sigmoid(1.5 * torch.randn((T, Hv), generator=g, device="cuda"))
        slots = R + 2
        s["state"] = 0.1 * torch.randn((slots, Hv, Dv, Dk), generator=g, device="cuda")
        s["slot"] = i32(torch.randperm(slots, generator=g, device="cuda")[:R])
        s["length"] = i32(_lengths(c)) if c["ragged"] else None
        s["fresh"] = torch.ones(R, dtype=torch.uint8, device="cuda") if c["fresh"] else None
        s["out"] = torch.zeros((T, Hv, Dv), dtype=act, device="cuda")
    if own:  # the handles, tables and workspaces that a program keeps
        import moe_expert_step_gb300 as ms
        kind = {"bf16": ms.BF16, "f32": ms.F32}
        if c["op"] == "plan":
            s["dims"] = ms.KvDims(Hq=16, Hkv=2, D=128, page=c["page"], n_pages=s["n_pages"], max_pages=s["max_pages"])
            s["ws"] = ms.kv_workspace(s["dims"], c["R"], 1)
        elif c["op"] == "rotary":
            s["dims"] = ms.KvDims(Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], page=64, n_pages=1, max_pages=1,
                                  dtype=kind[c["dtype"]])
            scaling = dict(none=ms.ROTARY_PLAIN, linear=ms.ROTARY_LINEAR, rotations=ms.ROTARY_ROTATIONS,
                           dimensions=ms.ROTARY_DIMENSIONS)[c["scaling"]]
            low, high = RAMP[c["scaling"]]
            s["turns"] = ms.rotary_frequencies(c["rot"], c["base"], scaling=scaling, factor=FACTOR, original=ORIGINAL,
                                               low=low, high=high)
        else:
            s["dims"] = ms.DeltaDims(Hk=c["Hk"], Hv=c["Hv"], Dk=c["Dk"], Dv=c["Dv"], n_slots=c["R"] + 2,
                                     dtype=kind[c["dtype"]])
            s["ws"] = ms.delta_workspace(s["dims"], c["R"], c["n"])
    return s


def _frequencies(c):
    """Radians a position of each pair, in 64 bits."""
    rot, kind = c["rot"], c["scaling"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    freq = c["base"] ** (-2.0 * i / rot)
    low, high = RAMP[kind]
    if kind == "none":
        return freq
    if kind == "linear":
        return freq / FACTOR
    if kind == "rotations":  # by the turns within the original context
        keep = ((ORIGINAL * freq / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    else:  # by the index, between those of `high` and of `low` turns
        at = lambda turns: rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(c["base"]))  # noqa: E731
        lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return freq * keep + freq / FACTOR * (1 - keep)


# ------------------------------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    return {"plan": _plain_plan, "rotary": _plain_rotary, "delta": _plain_delta}[c["op"]](s, c)


def _plan_out(s):
    return dict(head=s["head_out"], table=s["table"], ring=s["ring"], new_len=s["new_len"], pos=s["pos"], slots=s["slots"])


def _delta_out(s, c):
    return dict(out=s["out"], state=s["state"]) if c["write"] else dict(out=s["out"])


def _run_own(s, c):
    import moe_expert_step_gb300 as ms
    if c["op"] == "plan":
        ms.kv_cache_plan(s["dims"], c["R"], s["kv_len"], s["n_new"], s["ring"], s["head"], s["head_out"], s["table"],
                         s["new_len"], s["pos"], s["ws"], slots=s["slots"])
        return _plan_out(s)
    if c["op"] == "rotary":
        Hq, Hkv = c["Hq"], c["Hkv"]
        ms.block_rotary(s["dims"], s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["pos"], s["turns"], s["q_out"],
                        s["k_out"], interleaved=c["interleaved"], mscale=_mscale(c))
        return dict(q=s["q_out"], k=s["k_out"])
    ms.block_delta_rule(s["dims"], c["R"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["out"], s["ws"],
                        state_out=s["state"] if c["write"] else None, slot=s["slot"], length=s["length"],
                        fresh=s["fresh"], scale=c["Dk"] ** -0.5, qk_eps=1e-6)
    return _delta_out(s, c)


def _plain_plan(s, c):
    page, n, n_pages, max_pages = c["page"], c["n"], s["n_pages"], s["max_pages"]
    L, m = s["kv_len"].long(), s["n_new"].long()
    first, count = s["head"].long()
    held, need = -(-L // page), -(-(L + m) // page)
    grow, drop = (need - held).clamp(min=0), (held - need).clamp(min=0)
    grow = torch.where(need <= max_pages, grow, 0)
    asked, back = grow.cumsum(0), drop.cumsum(0)
    served = (need <= max_pages) & ((grow == 0) | (asked <= count))
    i = torch.arange(max_pages, device="cuda")
    takes = served & (grow > 0)
    new = takes[:, None] & (i >= held[:, None]) & (i < need[:, None])
    place = (asked - grow - held)[:, None] + i
    old = s["table"].clone()
    s["table"].copy_(torch.where(new, s["ring"][(first + place) % n_pages], old))
    gone = (i >= need[:, None]) & (i < held[:, None])
    place = (first + count + (back - drop - need)[:, None] + i) % n_pages
    ring = torch.cat([s["ring"], s["ring"][:1]])  # what stays is written to a place behind the ring
    ring.scatter_(0, torch.where(gone, place, n_pages).reshape(-1), old.reshape(-1))
    s["ring"].copy_(ring[:-1])
    taken = torch.where(takes, asked, 0).amax()
    s["head_out"].copy_(torch.stack([(first + taken) % n_pages, count - taken + back[-1]]))
    s["new_len"].copy_(torch.where(served, L + m, L))
    j = torch.arange(n, device="cuda")
    live = served[:, None] & (j < m[:, None])
    pos = torch.where(live, L[:, None] + j, -1)
    s["pos"].copy_(pos)
    pages = torch.gather(s["table"].long(), 1, (pos // page).clamp(min=0))
    s["slots"].copy_(torch.where(live, pages * page + pos % page, -1))
    return _plan_out(s)


def _plain_rotary(s, c):
    Hq, Hkv, rot = c["Hq"], c["Hkv"], c["rot"]
    pos = s["pos"].reshape(-1)
    angle = pos.double()[:, None] * s["freq"]  # in 64 bits: far positions turn thousands of times
    cos, sin = (_mscale(c) * f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    live = (pos >= 0)[:, None, None]
    for name, x in (("q_out", s["qkv"][:, :Hq]), ("k_out", s["qkv"][:, Hq:Hq + Hkv])):
        x = x.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        s[name].copy_(torch.where(live, y.to(s[name].dtype), s[name]))
    return dict(q=s["q_out"], k=s["k_out"])


def _plain_delta(s, c):
    """Chunks of up to 64 tokens: the triangular system of each chunk is inverted row by row, for all
    chunks at once; only the states go from chunk to chunk."""
    R, n, Hk, Hv, Dk, Dv = c["R"], c["n"], c["Hk"], c["Hv"], c["Dk"], c["Dv"]
    C = min(n, 64)
    N = -(-n // C) * C
    t = torch.arange(n, device="cuda")
    live = t < s["length"].long()[:, None] if s["length"] is not None else torch.ones((R, n), dtype=torch.bool, device="cuda")

    def heads(x, H):  # [R * n, H, ...] -> [R, Hv, chunks, C, ...], zeros behind a request's tokens
        x = torch.where(live.view(R, n, *[1] * (x.dim() - 1)), x.float().view(R, n, *x.shape[1:]), 0.0)
        x = torch.cat([x, x.new_zeros((R, N - n, *x.shape[2:]))], 1)
        x = x.repeat_interleave(Hv // H, 2).transpose(1, 2)
        return x.reshape(R, Hv, N // C, C, *x.shape[3:])

    unit = lambda x: x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    q, k, v = unit(heads(s["q"], Hk)) * Dk ** -0.5, unit(heads(s["k"], Hk)), heads(s["v"], Hv)
    G, beta = heads(s["g"], Hv).double().cumsum(-1), heads(s["beta"], Hv)[..., None]  # differences of long sums
    decay = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0)).float().tril()
    A = (beta * (k @ k.transpose(-1, -2)) * decay).tril(-1)
    X = torch.eye(C, device="cuda").expand_as(A).clone()
    for i in range(1, C):
        X[..., i, :i] = -(A[..., i, None, :i] @ X[..., :i, :i]).squeeze(-2)
    since, left = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    u, w = X @ (beta * v), X @ (beta * since * k)
    seen, inner, kept = q * since, (q @ k.transpose(-1, -2)) * decay, k * left
    slot = s["slot"].long()
    S = s["state"][slot].transpose(-1, -2)
    if s["fresh"] is not None:
        S = torch.where(s["fresh"].bool()[:, None, None, None], 0.0, S)
    o = torch.empty_like(v)
    for i in range(N // C):
        new = u[:, :, i] - w[:, :, i] @ S
        o[:, :, i] = seen[:, :, i] @ S + inner[:, :, i] @ new
        S = S * since[:, :, i, -1:] + kept[:, :, i].transpose(-1, -2) @ new
    o = o.reshape(R, Hv, N, Dv)[:, :, :n].transpose(1, 2).reshape(R * n, Hv, Dv)
    s["out"].copy_(torch.where(live.view(R * n, 1, 1), o.to(s["out"].dtype), s["out"]))
    if c["write"]:
        s["state"][slot] = S.transpose(-1, -2)
    return _delta_out(s, c)


# ------------------------------------------------------------------------------------- definitions


def exact(case, seed):
    """What run() returns where it is computed numbers, from the definitions in 64 bits."""
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "plan":
        return None
    if c["op"] == "rotary":
        Hq, rot = c["Hq"], c["rot"]
        pos = s["pos"].reshape(-1).to(f64)
        turn = torch.polar(torch.full_like(s["freq"], _mscale(c)).expand(len(pos), -1), torch.outer(pos, s["freq"]))
        y = s["qkv"][:, :Hq + c["Hkv"]].to(f64)
        x = y[..., :rot].clone()
        pairs = x.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else x.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        y[..., :rot] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        y[pos < 0] = 0.0
        return dict(q=y[:, :Hq], k=y[:, Hq:])
    R, n, Hk, Hv, Dk, Dv = c["R"], c["n"], c["Hk"], c["Hv"], c["Dk"], c["Dv"]
    q, k, v = (s[x].to(f64).reshape(R, n, s[x].shape[1], s[x].shape[2]) for x in "qkv")
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    g, beta = s["g"].to(f64).view(R, n, Hv), s["beta"].to(f64).view(R, n, Hv)
    lengths = torch.tensor(_lengths(c), device="cuda")
    slot = s["slot"].long()
    S = s["state"][slot].to(f64)  # [R][Hv][Dv][Dk]
    if c["fresh"]:
        S = torch.zeros_like(S)
    out = torch.zeros((R, n, Hv, Dv), dtype=f64, device="cuda")
    to = torch.arange(Hv, device="cuda") // (Hv // Hk)
    for t in range(max(_lengths(c))):
        on = (t < lengths)[:, None]
        a, b = torch.where(on, torch.exp(g[:, t]), 1.0), torch.where(on, beta[:, t], 0.0)
        kt, qt = k[:, t, to], q[:, t, to]
        S = S * a[..., None, None]
        held = (S @ kt[..., None]).squeeze(-1)
        S = S + (b[..., None] * (v[:, t] - held))[..., None] * kt[..., None, :]
        out[:, t] = torch.where(on[..., None], (S @ qt[..., None]).squeeze(-1) * Dk ** -0.5, 0.0)
    pool = s["state"].to(f64)
    pool[slot] = S
    out = out.reshape(R * n, Hv, Dv)
    return dict(out=out, state=pool) if c["write"] else dict(out=out)


# ------------------------------------------------------------------------------------- work


def work(case):
    """Bytes: inputs read once, outputs written once.  Operations: plan one a token; rotary six a
    pair; delta those of the recurrence, 7 for each element of a state a token."""
    c = case
    if c["op"] == "plan":
        R, n = c["R"], c["n"]
        return dict(bytes=4 * (3 * R + 4 + 2 * R * n + 2 * R * -(-n // (2 * c["page"]))), flops=R * n)
    act = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotary":
        T = c["R"] * c["n"]
        live = T - (c["n"] // 8 if c["n"] >= 8 else 0)
        return dict(bytes=2 * live * (c["Hq"] + c["Hkv"]) * c["D"] * act + 4 * T + 4 * c["rot"],
                    flops=3 * live * (c["Hq"] + c["Hkv"]) * c["rot"])
    T, R = sum(_lengths(c)), c["R"]
    state = c["Hv"] * c["Dk"] * c["Dv"]
    rows = T * (act * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"]) + 8 * c["Hv"])
    return dict(bytes=rows + 4 * R * state * ((not c["fresh"]) + c["write"]), flops=7 * T * state)
