"""The operators that a serving loop runs around the decode path: prompts
through the gated delta rule, the quantised state cache, and the gated group
norm of the layers' outputs.  `run` computes them in their plain form, or with
`own` through the framework's entry points."""
import math

import torch

own = False

CHUNK = 64          # tokens per chunk of the plain form
BLOCK = 32          # values that share a scale in the state cache
TINY = 2.0 ** -100  # a block whose largest magnitude is below is stored as zeros


# ------------------------------------------------------------------ cases
def _prefill(name, heads, dk, dv, act, lens, batch, carried, packed=False):
    """lens: tokens of each prompt; carried: every carried-th prompt goes on
    from its sequence's state (0: none does); packed: q, k and v are slices of
    one projection's rows."""
    c = {"op": "prefill", "heads": heads, "dk": dk, "dv": dv, "act": act, "lens": ",".join(map(str, lens)),
         "batch": batch, "carried": carried, "packed": packed}
    return dict(c, name=name) if name else c


def _cache(name, family, heads, dk, dv, bits, n):
    c = {"op": "cache", "family": family, "heads": heads, "dk": dk, "dv": dv, "bits": bits, "n": n}
    return dict(c, name=name) if name else c


def _norm(name, rows, groups, width, act, form):
    """form: "rms-silu" (the delta-rule layers' output), "gate-first" (Mamba-2's),
    "centred" (group norm with weight, bias and SiLU, no gate)."""
    c = {"op": "norm", "rows": rows, "groups": groups, "width": width, "act": act, "form": form}
    return dict(c, name=name) if name else c


RAGGED = [1, 2048, 17, 700, 64, 1500, 3, 0, 333, 1024, 65, 2500, 129, 8, 911, 1777, 256, 640, 31, 1200, 63, 480, 2222, 90]


def listed():
    return [
        # a decode batch that takes its tokens through the prompt path (every state is read and written)
        _prefill("step_b256", 32, 128, 128, "bf16", [1] * 256, 256, 1),
        # drafted tokens of 48 sequences checked at once
        _prefill("draft_b48", 32, 128, 128, "bf16", [5] * 48, 64, 1),
        # one short prompt alone: latency
        _prefill("one_short", 32, 128, 128, "bf16", [517], 4, 0, True),
        # one long prompt alone: the few rows that a long axis leaves
        _prefill("one_long", 32, 128, 128, "bf16", [16384], 2, 0),
        # a prompt batch as a scheduler makes it: ragged, some continued, slices of one projection
        _prefill("ragged_24", 32, 128, 128, "bf16", RAGGED, 32, 3, True),
        # small heads held in 32 bits
        _prefill("f32_heads64", 16, 64, 64, "f32", [300, 1, 77, 512, 129, 40, 256, 333], 8, 2),
        # a delta-rule layer's sequences parked in 8 bits and read back into other rows
        _cache("park8_gdn", "gdn", 32, 128, 128, 8, 128),
        # a Mamba-2 layer's in 4 bits
        _cache("park4_m2", "mamba2", 128, 128, 64, 4, 96),
        # one sequence: latency
        _cache("park8_one", "gdn", 32, 128, 128, 8, 1),
        # the outputs of a prompt batch, normalised by head and gated
        _norm("norm_prompt", 16384, 32, 128, "bf16", "rms-silu"),
        # a decode step of the batch-320 Mamba-2 layer: 8 groups of 1024 channels, gated first
        _norm("norm_step_m2", 320, 8, 1024, "bf16", "gate-first"),
        # centred group norm in 32 bits
        _norm("norm_centred", 2049, 16, 64, "f32", "centred"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "cache", "norm"))
    if op == "prefill":
        dk, dv = rng.choice(((128, 128), (128, 128), (128, 64), (64, 64)))
        act = rng.choice(("bf16", "bf16", "bf16", "f32"))
        heads = rng.randint(2, 32)
        n = _log(rng, 1, 64)
        top = (12000 if act == "bf16" else 2500) // n
        hi = _log(rng, 1, top)
        lens = [rng.randint(0, hi) for _ in range(n - 1)] + [max(1, hi)]
        rng.shuffle(lens)
        return _prefill(None, heads, dk, dv, act, lens, n + rng.randint(0, 8), rng.randint(0, 3), rng.random() < 0.5)
    if op == "cache":
        family = rng.choice(("gdn", "kda", "mamba2"))
        dk, dv = rng.choice(((128, 128), (128, 64), (64, 64)))
        return _cache(None, family, rng.choice((8, 16, 32, 48)), dk, dv, rng.choice((8, 4)), _log(rng, 1, 120))
    form = rng.choice(("rms-silu", "gate-first", "centred"))
    width = 8 * _log(rng, 4, 256)
    groups = rng.randint(1, max(1, min(40, 8192 // width)))
    return _norm(None, _log(rng, 1, (1 << 26) // (width * groups)), groups, width, rng.choice(("bf16", "f32")), form)


# ----------------------------------------------------------------- inputs
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ranks(heads, dk):
    """Sketch ranks of the heads: 2 to min(16, dk), about 8 on average."""
    return [min(dk, 2 + (5 * h) % 13) for h in range(heads)]


def _offsets(heads, dk):
    off = [0]
    for r in _ranks(heads, dk):
        off.append(off[-1] + r)
    return off


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _has_state(case):
    n = len(_lens(case))
    return [int(case["carried"] > 0 and i % case["carried"] == 0) for i in range(n)]


def _layer(case, family, batch, act, off):
    """The framework's layer with its buffers."""
    import numpy as np
    from ssm_decode_amd.layer import DecodeLayer
    H = case["heads"]
    groups = H // 8 if family == "mamba2" else H
    return DecodeLayer(family, batch, H, groups, case["dk"], case["dv"], 16, act, act, np.array(off))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    st = {"case": case}
    if case["op"] == "norm":
        rows, G, W, dt = case["rows"], case["groups"], case["width"], DT[case["act"]]
        st["x"] = (normal(rows, G, W) + (0.5 if case["form"] == "centred" else 0.0)).to(dt)
        st["weight"] = 1.0 + 0.1 * normal(G, W)
        st["bias"] = 0.1 * normal(G, W) if case["form"] == "centred" else None
        st["gate"] = None if case["form"] == "centred" else normal(rows, G, W).to(dt)
        if own:
            from ssm_decode_amd.serving import OutputNorm
            st["norm"] = OutputNorm(st["weight"], st["bias"], eps=1e-5, act="silu", centred=case["form"] == "centred",
                                    gate_first=case["form"] == "gate-first")
            st["y"] = torch.empty_like(st["x"])
        return st

    H, dk, dv = case["heads"], case["dk"], case["dv"]
    off = _offsets(H, dk)
    R = off[-1]
    P = normal(R, dk) / math.sqrt(dk)
    st["P_heads"] = torch.zeros(H, 16, dk, device="cuda")
    st["rows"] = torch.tensor([16 * h + j for h, r in enumerate(_ranks(H, dk)) for j in range(r)], device="cuda")
    st["P_heads"].view(-1, dk)[st["rows"]] = P
    if case["op"] == "cache":
        n = case["n"]
        # heads of different sizes, and values that are not all alike within a block
        S = normal(2 * n, H, dk, dv) * (0.02 + uniform(2 * n, H, dk, 1))
        st.update(n=n, off=off, P=P, S=S)
        st["src"] = torch.arange(n, device="cuda", dtype=torch.int32)
        st["dst"] = torch.arange(2 * n - 1, n - 1, -1, device="cuda", dtype=torch.int32)
        st["slots"] = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        if own:
            from ssm_decode_amd.serving import StateCache
            lay = _layer(case, case["family"], 2 * n, "bf16", off)
            lay.S.copy_(S)
            lay.Pt.copy_(P)
            st.update(layer=lay, cache=StateCache(lay, n, case["bits"]), S=None)
        else:
            st["U"] = torch.zeros(2 * n, R, dv, device="cuda", dtype=torch.bfloat16)
        return st

    lens, dt, batch = _lens(case), DT[case["act"]], case["batch"]
    n, N = len(lens), sum(lens)
    q = normal(N, H, dk)
    k = normal(N, H, dk)
    q = (q / q.norm(dim=-1, keepdim=True)).to(dt)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    v = (normal(N, H, dv) / math.sqrt(dv)).to(dt)
    if case["packed"]:
        rows = torch.cat([q.reshape(N, -1), k.reshape(N, -1), v.reshape(N, -1)], dim=1)
        q = rows[:, :H * dk].unflatten(1, (H, dk))
        k = rows[:, H * dk:2 * H * dk].unflatten(1, (H, dk))
        v = rows[:, 2 * H * dk:].unflatten(1, (H, dv))
    st.update(q=q, k=k, v=v, gate=0.9 + 0.1 * uniform(N, H), beta=uniform(N, H), lens=lens, off=off, P=P)
    S = 0.1 * normal(batch, H, dk, dv)
    start = [0]
    for x in lens:
        start.append(start[-1] + x)
    st["start"] = torch.tensor(start, device="cuda", dtype=torch.int32)
    # the prompts' sequences, spread over the batch in another order
    st["seqs"] = torch.randperm(batch, generator=g, device="cuda")[:n].to(torch.int32)
    st["has_state"] = torch.tensor(_has_state(case), device="cuda", dtype=torch.int32)
    # where each prompt's tokens lie in a rectangle of whole chunks
    C = min(CHUNK, max(lens))
    L = -(-max(lens) // C) * C
    col = torch.arange(L, device="cuda")
    ln = torch.tensor(lens, device="cuda")[:, None]
    st["there"] = col[None] < ln
    st["token"] = torch.where(st["there"], st["start"][:-1, None].long() + col[None], 0)
    st["C"] = C
    if own:
        from ssm_decode_amd.serving import Prompts
        lay = _layer(case, "gdn", batch, case["act"], off)
        lay.S.copy_(S)
        lay.Pt.copy_(P)
        st["layer"] = lay
        st["prompts"] = Prompts(lay, q, k, v, st["gate"], st["beta"], torch.empty(N, H, dv, device="cuda", dtype=dt),
                                st["start"], seqs=st["seqs"], has_state=st["has_state"])
    else:
        st["S"] = S
        st["U"] = torch.zeros(batch, R, dv, device="cuda", dtype=dt)
    return st


# ------------------------------------------------------------- plain forms
def _sketch(S, st):
    """U rows: u_j = S_h^T p_j for every row j of every head h."""
    U = torch.matmul(st["P_heads"], S)          # [n][H][16][dv], the rows that a head lacks as zeros
    return U.flatten(1, 2)[:, st["rows"]]


def _plain_prefill(st):
    case = st["case"]
    H, dk, dv, C = case["heads"], case["dk"], case["dv"], st["C"]
    tok, there = st["token"], st["there"]
    n, L = tok.shape
    X = L // C

    def chunks(x, fill):
        """[tokens][H][...] -> [chunks][n H][C][...] in 32 bits, filled behind each prompt's end."""
        y = x[tok].float()
        y = torch.where(there.reshape(n, L, *([1] * (y.dim() - 2))), y, torch.full_like(y[:1, :1], fill))
        y = y.transpose(1, 2).reshape(n * H, X, C, *y.shape[3:])
        return y.transpose(0, 1).contiguous()

    q, k, v = chunks(st["q"], 0.0), chunks(st["k"], 0.0), chunks(st["v"], 0.0)
    al, be = chunks(st["gate"], 1.0), chunks(st["beta"], 0.0)
    g = al.cumprod(-1)
    # D[i][j] = product of the decays after j up to i
    low = torch.tril(torch.ones(C, C, device=al.device, dtype=torch.bool))
    D = torch.where(torch.tril(low, -1), al[..., :, None], torch.ones_like(al[..., :, None])).cumprod(-2) * low
    A = be[..., :, None] * D * torch.matmul(k, k.transpose(-1, -2).contiguous()) * torch.tril(low, -1)
    T = torch.zeros_like(A)
    for i in range(C):      # forward substitution, every chunk at once
        T[..., i, :] = -torch.matmul(A[..., i:i + 1, :i], T[..., :i, :])[..., 0, :] if i else 0.0
        T[..., i, i] = 1.0
    T = T * be[..., None, :]
    M = D * torch.matmul(q, k.transpose(-1, -2).contiguous())
    kT = k.transpose(-1, -2).contiguous()
    rows = st["seqs"].long()
    S = torch.where(st["has_state"].reshape(n, 1, 1, 1) != 0, st["S"][rows], torch.zeros_like(st["S"][rows]))
    S = S.reshape(n * H, dk, dv)
    o = torch.empty(X, n * H, C, dv, device=S.device)
    for c in range(X):      # from chunk to chunk
        u = torch.matmul(T[c], v[c] - g[c][..., None] * torch.matmul(k[c], S))
        o[c] = g[c][..., None] * torch.matmul(q[c], S) + torch.matmul(M[c], u)
        S = g[c][:, -1, None, None] * S + torch.matmul(kT[c], D[c][:, -1, :, None] * u)
    S = S.reshape(n, H, dk, dv)
    st["S"][rows] = S
    o = o.reshape(X, n, H, C, dv).permute(1, 0, 3, 2, 4).reshape(n, L, H, dv)[there]
    st["U"][rows] = _sketch(S, st).to(st["U"].dtype)
    return {"o": o.to(st["q"].dtype), "S": st["S"], "U": st["U"]}


def _plain_cache(st):
    n, case = st["n"], st["case"]
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    top = 127.0 if case["bits"] == 8 else 7.0
    held_scale = torch.empty(n, H, dk, dv // BLOCK, 1, device="cuda")
    held = torch.empty(n, H, dk, dv // BLOCK, BLOCK, device="cuda", dtype=torch.int8)
    src, dst, slots = st["src"].long(), st["dst"].long(), st["slots"].long()
    x = st["S"][src].reshape(n, H, dk, dv // BLOCK, BLOCK)
    amax = x.abs().amax(-1, keepdim=True)
    scale = torch.where(amax >= TINY, (amax.double() / top).float(), torch.zeros_like(amax))
    code = torch.round(x.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double())
    code = torch.where(scale > 0, code, torch.zeros_like(code))
    held[slots] = code.to(torch.int8)
    held_scale[slots] = scale
    S = (held[slots].float() * held_scale[slots]).reshape(n, H, dk, dv)
    st["S"][dst] = S
    st["U"][dst] = _sketch(S, st).to(st["U"].dtype)
    return {"S": st["S"], "U": st["U"]}


def _plain_norm(st):
    x, form = st["x"].float(), st["case"]["form"]
    z = st["gate"]
    if z is not None:
        z = z.float()
        z = z / (1.0 + torch.exp(-z))
    if form == "gate-first":
        x = x * z
    if form == "centred":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * st["weight"]
    if form == "centred":
        y = y + st["bias"]
        y = y / (1.0 + torch.exp(-y))
    elif form == "rms-silu":
        y = y * z
    return {"y": y.to(st["x"].dtype)}


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"prefill": _plain_prefill, "cache": _plain_cache, "norm": _plain_norm}[op](st)
    if op == "prefill":
        lay, pr = st["layer"], st["prompts"]
        lay.prefill(pr)
        return {"o": pr.o, "S": lay.S, "U": lay.U}
    if op == "cache":
        lay = st["layer"]
        lay.save_state(st["cache"], st["src"], st["slots"])
        lay.load_state(st["cache"], st["dst"], st["slots"])
        return {"S": lay.S, "U": lay.U}
    from ssm_decode_amd.serving import group_norm
    group_norm(st["x"], st["norm"], st["y"], gate=st["gate"])
    return {"y": st["y"]}


# ---------------------------------------------------------- 64-bit values
def _at(rows, n, x):
    """x in the given rows of n, zeros in the others."""
    y = torch.zeros(n, *x.shape[1:], device=x.device, dtype=x.dtype)
    y[rows.long()] = x
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        x = st["x"].double()
        z = None if st["gate"] is None else st["gate"].double()
        if case["form"] == "gate-first":
            x = x * (z * torch.sigmoid(z))
        mean = x.mean(-1, keepdim=True) if case["form"] == "centred" else 0.0
        var = ((x - mean) ** 2).mean(-1, keepdim=True)
        y = (x - mean) * torch.rsqrt(var + 1e-5) * st["weight"].double()
        if case["form"] == "centred":
            y = y + st["bias"].double()
            y = y * torch.sigmoid(y)
        elif case["form"] == "rms-silu":
            y = y * z * torch.sigmoid(z)
        return {"y": y}
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    P, off = st["P"].double(), st["off"]

    def sketch(S):
        return torch.cat([torch.stack([(S[:, h] * P[j][:, None]).sum(1) for j in range(off[h], off[h + 1])], dim=1)
                          for h in range(H)], dim=1)

    if case["op"] == "cache":
        S = st["S"].double()
        top = 127 if case["bits"] == 8 else 7
        x = S[st["src"].long()].unflatten(-1, (-1, BLOCK))
        amax = x.abs().amax(-1, keepdim=True)
        s = (amax / top).float().double()       # the scale is held in 32 bits
        live = amax >= TINY
        back = torch.where(live, torch.round(x / torch.where(live, s, torch.ones_like(s))) * s, torch.zeros_like(x)).flatten(-2)
        S[st["dst"].long()] = back
        return {"S": S, "U": _at(st["dst"], len(S), sketch(back))}
    # the recurrence, token by token, every prompt and head at once
    rows = st["seqs"].long()
    S0 = st["S"].double()
    S = S0[rows] * st["has_state"].double()[:, None, None, None]
    o = torch.zeros(sum(st["lens"]), H, dv, device="cuda", dtype=torch.float64)
    order = sorted(range(len(st["lens"])), key=lambda i: -st["lens"][i])
    S = S[order]
    first = st["start"].long()[order]
    for t in range(max(st["lens"])):
        m = sum(x > t for x in st["lens"])      # the prompts that still have a token: the longest come first
        at = first[:m] + t
        k, q, v = st["k"][at].double(), st["q"][at].double(), st["v"][at].double()
        a, b = st["gate"][at].double()[..., None], st["beta"][at].double()[..., None]
        s = S[:m]
        s.mul_(a[..., None])
        u = b * (v - torch.matmul(k[:, :, None], s)[:, :, 0])
        s.addcmul_(k[..., None], u[:, :, None])
        o[at] = torch.matmul(q[:, :, None], s)[:, :, 0]
    back = torch.empty_like(S)
    back[order] = S
    S0[rows] = back
    return {"o": o, "S": S0, "U": _at(st["seqs"], len(S0), sketch(back))}


# ------------------------------------------------------------------- work
def work(case):
    size = 2 if case.get("act", "bf16") == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["groups"] * case["width"]
        streams = 2 if case["form"] == "centred" else 3
        return {"bytes": n * size * streams, "flops": 12 * n}
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    R = sum(_ranks(H, dk))
    if case["op"] == "cache":
        n, state = case["n"], case["heads"] * dk * dv
        held = state * case["bits"] / 8 + state / BLOCK * 4
        return {"bytes": n * (8 * state + 2 * held + R * dv * 2) + R * dk * 4, "flops": n * (6 * state + 2 * R * dk * dv)}
    lens, N = _lens(case), sum(_lens(case))
    read = sum(_has_state(case))
    state = H * dk * dv
    return {"bytes": N * H * ((2 * dk + 2 * dv) * size + 8) + 4 * state * (read + len(lens)) + len(lens) * R * dv * size + R * dk * 4,
            "flops": N * H * 6 * dk * dv + len(lens) * 2 * R * dk * dv}
