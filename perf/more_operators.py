"""Cases, plain forms and 64-bit values of a state space layer's operators over state slots.

A layer of a state space model is, between its two projections, three operators:

short convolution ("conv") -- per channel c a causal filter of `width` taps over the tokens,
    o_t = silu(bias + sum_j w[j] u_{t - width + 1 + j}),
  which reads the last width - 1 inputs of the request's earlier tokens from its slot and
  leaves the newest there.

selective scan ("scan") -- per head a state S [p, n]; with dt' = softplus(dt + dt_bias) a token does
    S <- exp(dt' A) S + (dt' x) B^T;  o = S C + D x.
  Head h reads B and C of group h // (heads / groups).

gated norm ("norm") -- o = rms(u) w over groups of columns, u = o_scan silu(z), or
  o = rms(o_scan) w silu(z) with the gate after the norm.

The scan and the convolution run as one token for each of many slots ("decode"), as a few
tokens for each of them with what a slot holds after every token kept ("multi", the pass that
checks a draft), and over whole prompts packed back to back ("prefill").

`run` computes the plain forms, or calls the library where `own` is set.
"""
import math
import random

import torch

own = False

EPS = 1e-5  # of the norms


# ------------------------------------------------------------------------------ cases

def _scan(op, name, heads, n, tokens=1, ragged=False, state="f32", inputs="bf16", out="bf16"):
    h, g, p, ds = heads
    return {"name": name, "kind": "scan", "op": op, "heads": h, "groups": g, "p": p, "ds": ds, "n": n, "tokens": tokens,
            "ragged": ragged, "state": state, "inputs": inputs, "out": out}


def _conv(op, name, channels, n, tokens=1, ragged=False, width=4, inputs="bf16", bias=True):
    return {"name": name, "kind": "conv", "op": op, "channels": channels, "n": n, "tokens": tokens, "ragged": ragged,
            "width": width, "inputs": inputs, "bias": bias}


def _norm(name, rows, groups, size, first, x="bf16", z="bf16", out="bf16"):
    return {"name": name, "kind": "norm", "op": "norm", "rows": rows, "groups": groups, "size": size, "first": first,
            "x": x, "z": z, "out": out}


MANY = (64, 1, 64, 128)     # one B and C for all heads
GROUPED = (32, 8, 64, 128)
BROAD = (16, 2, 128, 128)
SMALL = (24, 1, 64, 64)


def listed():
    return [
        # one user's next token at one layer: latency
        _scan("decode", "scan_one", MANY, 1),
        # a full serving batch at one layer
        _scan("decode", "scan_batch", MANY, 256),
        # states kept in bf16, float32 inputs and outputs
        _scan("decode", "scan_small_states", SMALL, 203, state="bf16", inputs="f32", out="f32"),
        # the pass over a draft of 4, with the five states to go back to
        _scan("multi", "scan_check", GROUPED, 48, tokens=5, out="f32"),
        # a short prompt that no tile divides
        _scan("prefill", "scan_short", MANY, 1, tokens=93, out="f32"),
        # prompts of a mixed serving step: 64 sequences of 1 to 1,023 tokens
        _scan("prefill", "scan_ragged", GROUPED, 64, tokens=512, ragged=True),
        # one long document, few heads, states kept in bf16: little runs side by side
        _scan("prefill", "scan_long", BROAD, 1, tokens=16383, state="bf16", out="f32"),
        # long prompts of a few users
        _scan("prefill", "scan_8x4096", MANY, 8, tokens=4096),
        # a serving batch's next tokens: x, B and C of one layer
        _conv("decode", "conv_batch", 4352, 256),
        # prompts of a mixed serving step
        _conv("prefill", "conv_ragged", 4096, 64, tokens=512, ragged=True),
        # a serving batch's rows, the norm over the whole row
        _norm("norm_batch", 256, 1, 4096, True),
        # 32,768 tokens' heads, the gate after the norm
        _norm("norm_heads", 32768, 32, 128, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_any(rng):
    kind = rng.choice(("scan", "scan", "conv", "norm"))
    op = rng.choice(("decode", "multi", "prefill", "prefill"))
    inputs, out = rng.choice(("bf16", "bf16", "f32")), rng.choice(("bf16", "f32"))
    if kind == "norm":
        groups, size = rng.choice(((1, 8 * _log_int(rng, 1, 1100)), (8, 8 * rng.randint(8, 130)), (32, 128), (64, 64)))
        c = _norm("", _log_int(rng, 1, 32768), groups, size, rng.random() < 0.5, x=rng.choice(("bf16", "f32")), z=inputs, out=out)
    else:
        n = _log_int(rng, 1, {"decode": 300, "multi": 64, "prefill": 64}[op])
        tokens = 1 if op == "decode" else rng.randint(2, 9) if op == "multi" else _log_int(rng, 1, max(2, 32768 // n // 2))
        ragged = op == "prefill" and rng.random() < 0.5
        if kind == "conv":
            c = _conv(op, "", 8 * _log_int(rng, 8, 800), n, tokens, ragged, width=rng.choice((2, 3, 4, 4)), inputs=inputs,
                      bias=rng.random() < 0.7)
        else:
            heads = rng.choice((MANY, GROUPED, BROAD, SMALL, (6, 3, 128, 64), (5, 1, 64, 128)))
            c = _scan(op, "", heads, n, tokens, ragged, state=rng.choice(("f32", "f32", "bf16")),
                      inputs="bf16" if op == "prefill" else inputs, out=out)
    del c["name"]
    return c


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["kind"], (0, 0))
        most[c["kind"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        c = _draw_any(rng)
        w = work(c)
        if w["bytes"] <= most[c["kind"]][0] and w["flops"] <= most[c["kind"]][1]:
            return c


def lengths(case):
    """The sequences' lengths: all alike, or spread over 1 .. 2 tokens - 1 (the same for every seed)."""
    n, t = case["n"], case["tokens"]
    if not case["ragged"]:
        return [t] * n
    rng = random.Random(n * 100003 + t)
    return [rng.randint(1, max(1, 2 * t - 1)) for _ in range(n)]


def _rows(case):
    return sum(lengths(case)) if case["op"] == "prefill" else case["n"] * case["tokens"]


_BYTES = {"bf16": 2, "f32": 4}


def work(case):
    if case["kind"] == "norm":
        cells = case["rows"] * case["groups"] * case["size"]
        return {"bytes": float(cells * (_BYTES[case["x"]] + _BYTES[case["z"]] + _BYTES[case["out"]])), "flops": 8.0 * cells}
    rows, e = _rows(case), _BYTES[case["inputs"]]
    if case["kind"] == "conv":
        ch, w = case["channels"], case["width"]
        held = ch * (w - 1) * e
        kept = rows * held if case["op"] == "multi" else 0
        return {"bytes": float(2 * rows * ch * e + 2 * case["n"] * held + kept + ch * w * e), "flops": (2.0 * w + 4) * rows * ch}
    h, p, ds = case["heads"], case["p"], case["ds"]
    est = _BYTES[case["state"]]
    per_row = (h * p + 2 * case["groups"] * ds + h) * e + h * p * _BYTES[case["out"]]
    states = case["n"] * h * p * ds * est
    kept = rows * h * p * ds * est if case["op"] == "multi" else 0
    return {"bytes": float(rows * per_row + 2 * states + kept), "flops": 5.0 * rows * h * p * ds}


# ----------------------------------------------------------------------------- inputs

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(seed, dev):
    return torch.Generator(device=dev).manual_seed(int(seed) * 6151 + 29)


def _slots(case, s, gen, dev):
    """Which slots the rows or sequences use, and where the sequences lie."""
    n, t = case["n"], case["tokens"]
    s["slots"] = n + 3
    s["ids"] = torch.randperm(n + 3, device=dev, generator=gen)[:n].to(torch.int32)
    if case["op"] == "multi":
        s["snap_ids"] = torch.randperm(n * t, device=dev, generator=gen).to(torch.int32).view(n, t)
    if case["op"] == "prefill":
        lens = torch.tensor(lengths(case), device=dev)
        s["cu"] = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
        s["longest"] = max(lengths(case))


def _scan_inputs(case, seed):
    """x, B and C side by side as the convolution leaves them (after its SiLU), dt as a column range of
    the projection; A in -16 .. -1 and a dt_bias whose softplus spreads over 0.001 .. 0.1."""
    dev = _device()
    gen = _gen(seed, dev)
    h, g, p, ds, rows = case["heads"], case["groups"], case["p"], case["ds"], _rows(case)
    kind = _TYPES[case["inputs"]]
    u = torch.randn(rows, h * p + 2 * g * ds, device=dev, generator=gen)
    xbc = torch.nn.functional.silu(u).to(kind)
    del u
    s = {"case": case, "xbc": xbc}
    s["x"] = xbc[:, : h * p].unflatten(1, (h, p))
    s["b"] = xbc[:, h * p: h * p + g * ds].unflatten(1, (g, ds))
    s["c"] = xbc[:, h * p + g * ds:].unflatten(1, (g, ds))
    s["dt"] = (torch.randn(rows, 24 + h, device=dev, generator=gen) * 0.7).to(kind)[:, 24:]
    s["A"] = -(1.0 + 15.0 * torch.rand(h, device=dev, generator=gen))
    dt = torch.exp(torch.rand(h, device=dev, generator=gen) * math.log(100.0) + math.log(1e-3))
    s["bias"] = dt + torch.log(-torch.expm1(-dt))     # softplus(bias) = dt
    s["D"] = torch.randn(h, device=dev, generator=gen) * 0.5 + 1.0
    _slots(case, s, gen, dev)
    s["states"] = (torch.randn(s["slots"], 1, h, p, ds, device=dev, generator=gen) * 0.1).to(_TYPES[case["state"]])
    if case["op"] == "multi":
        for name in ("x", "b", "c", "dt"):
            s[name] = s[name].unflatten(0, (case["n"], case["tokens"]))
        s["snaps"] = torch.zeros(case["n"] * case["tokens"], 1, h, p, ds, device=dev, dtype=_TYPES[case["state"]])
    return s


def _conv_inputs(case, seed):
    """A column range of the projection's output, and the filters of a trained layer's size."""
    dev = _device()
    gen = _gen(seed, dev)
    ch, w, rows, kind = case["channels"], case["width"], _rows(case), _TYPES[case["inputs"]]
    wide = torch.randn(rows, ch + 64, device=dev, generator=gen).to(kind)
    s = {"case": case, "u": wide[:, 64:]}
    s["w"] = ((torch.rand(ch, w, device=dev, generator=gen) * 2 - 1) * w ** -0.5).to(kind)
    s["bias"] = (torch.randn(ch, device=dev, generator=gen) * 0.2).to(kind) if case["bias"] else None
    _slots(case, s, gen, dev)
    s["tails"] = torch.randn(s["slots"], 1, w - 1, ch, device=dev, generator=gen).to(kind)
    if case["op"] == "multi":
        s["u"] = s["u"].unflatten(0, (case["n"], case["tokens"]))
        s["snaps"] = torch.zeros(case["n"] * case["tokens"], 1, w - 1, ch, device=dev, dtype=kind)
    return s


def _norm_inputs(case, seed):
    """A scan's outputs, and the gate as a column range of the projection."""
    dev = _device()
    gen = _gen(seed, dev)
    rows, width = case["rows"], case["groups"] * case["size"]
    s = {"case": case}
    s["x"] = (torch.randn(rows, width, device=dev, generator=gen) * 0.8).to(_TYPES[case["x"]])
    s["z"] = torch.randn(rows, width + 64, device=dev, generator=gen).to(_TYPES[case["z"]])[:, :width]
    s["w"] = (1.0 + 0.1 * torch.randn(width, device=dev, generator=gen)).to(torch.bfloat16)
    return s


_INPUTS = {"scan": _scan_inputs, "conv": _conv_inputs, "norm": _norm_inputs}


def prepare(case, seed):
    case = dict(case)
    s = _INPUTS[case["kind"]](case, seed)
    if own and case["kind"] != "norm":  # the same contents, in the pool that a server keeps them in
        from rwkv_wkv_gb300 import SsmPool
        kept = len(s["snaps"]) if "snaps" in s else 0
        if case["kind"] == "scan":
            pool = SsmPool(1, case["heads"], case["groups"], s["slots"], n_snapshots=kept, head_p=case["p"],
                           d_state=case["ds"], state_dtype=case["state"], out_dtype=case["out"])
            held, snaps = pool.states, pool.snapshots
        else:
            pool = SsmPool(1, 1, 1, s["slots"], n_snapshots=kept, head_p=64, d_state=64, conv_channels=case["channels"],
                           conv_width=case["width"], conv_dtype=case["inputs"])
            held, snaps = pool.conv_tails, pool.conv_snapshots
        name = "states" if case["kind"] == "scan" else "tails"
        held.copy_(s[name])
        s["pool"], s[name] = pool, held
        if kept:
            snaps.zero_()
            s["snaps"] = snaps
    return s


# -------------------------------------------------------------------------- one pass

def _steps(s):
    """dt' of each token and head, in float32."""
    return torch.nn.functional.softplus(s["dt"].float() + s["bias"], threshold=20.0)


def _per_head(x, case):
    return x.float().repeat_interleave(case["heads"] // case["groups"], dim=-2)


def _token(s, state, x, b, c, dt):
    """One token of each row: state [rows, h, p, ds]; x [rows, h, p]; b, c [rows, h, ds]; dt [rows, h]."""
    state = state * torch.exp(dt * s["A"])[..., None, None] + (dt[..., None] * x)[..., None] * b[..., None, :]
    return state, (state * c[..., None, :]).sum(-1) + s["D"][:, None] * x


def _scan_tokens(s):
    case, at = s["case"], s["ids"].long()
    x, b, c, dt = s["x"].float(), _per_head(s["b"], case), _per_head(s["c"], case), _steps(s)
    state = s["states"][at, 0].float()
    out = _TYPES[case["out"]]
    if case["op"] == "decode":
        state, o = _token(s, state, x, b, c, dt)
        s["states"][at, 0] = state.to(s["states"].dtype)
        return {"o": o.to(out), "states": s["states"]}
    o = torch.empty(x.shape, device=x.device, dtype=out)
    for t in range(case["tokens"]):
        state, ot = _token(s, state, x[:, t], b[:, t], c[:, t], dt[:, t])
        o[:, t] = ot.to(out)
        state = state.to(s["snaps"].dtype)      # what a step stores is what the next one reads
        s["snaps"][s["snap_ids"][:, t].long(), 0] = state
        state = state.float()
    s["states"][at, 0] = state.to(s["states"].dtype)
    return {"o": o, "states": s["states"], "snapshots": s["snaps"]}


CHUNK = 64


def _scan_prefill(s):
    """By chunks of 64 tokens.  With L_t the running sum of dt' A inside a chunk,
        O = diag(exp L) C S^T + (C B^T * exp(L_t - L_s) dt'_s, s <= t) X + D X,
        S <- exp(L_end) S + (diag(dt' exp(L_end - L)) X)^T B."""
    case, dev = s["case"], s["x"].device
    chunks = max(1, -(-s["longest"] // CHUNK))
    lens = s["cu"].diff().long()
    pos = torch.arange(chunks * CHUNK, device=dev)
    live = pos[None] < lens[:, None]                                    # the padding is tokens that change nothing
    at = torch.where(live, s["cu"][:-1].long()[:, None] + pos[None], 0)

    def chunked(x):  # [rows, heads, ...] -> [n, heads, chunks, 64, ...]
        x = x[at].float()
        x = torch.where(live.view(*live.shape, *([1] * (x.dim() - 2))), x, 0.0)
        return x.transpose(1, 2).unflatten(2, (chunks, CHUNK))

    x, b, c, dt = chunked(s["x"]), chunked(s["b"]), chunked(s["c"]), chunked(_steps(s))
    share = case["heads"] // case["groups"]
    total = (dt * s["A"][:, None, None]).double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    score = c @ b.transpose(-1, -2)
    state = s["states"][s["ids"].long(), 0].float()
    o = torch.empty_like(x)
    for k in range(chunks):
        run, d, xk = total[:, :, k], dt[:, :, k], x[:, :, k]
        bk, ck = b[:, :, k].repeat_interleave(share, 1), c[:, :, k].repeat_interleave(share, 1)
        decay = torch.where(low, run[..., :, None] - run[..., None, :], -math.inf).exp().float()
        inside = decay * d[..., None, :] * score[:, :, k].repeat_interleave(share, 1)
        o[:, :, k] = run.exp().float()[..., None] * (ck @ state.transpose(-1, -2)) + inside @ xk
        left = (run[..., -1:] - run).exp().float() * d
        state = run[..., -1].exp().float()[..., None, None] * state + (left[..., None] * xk).transpose(-1, -2) @ bk
    o = o + s["D"][:, None, None, None] * x
    s["states"][s["ids"].long(), 0] = state.to(s["states"].dtype)
    return {"o": o.flatten(2, 3).transpose(1, 2)[live].to(_TYPES[case["out"]]), "states": s["states"]}


def _plain_conv(s):
    case = s["case"]
    w, ids, dev = case["width"], s["ids"].long(), s["u"].device
    kind = s["u"].dtype
    if case["op"] == "prefill":
        rows = s["u"]
        start = s["cu"][:-1].long()
        lens = s["cu"].diff().long()
    else:
        rows = s["u"].flatten(0, 1) if case["op"] == "multi" else s["u"]
        start = torch.arange(case["n"], device=dev) * case["tokens"]
        lens = torch.full_like(start, case["tokens"])
    # each request's tail and then its tokens, one request after the other
    n, total = case["n"], len(rows)
    first = start + (w - 1) * torch.arange(n, device=dev)              # of its tail
    seq = torch.repeat_interleave(torch.arange(n, device=dev), lens, output_size=total)
    own_at = torch.arange(total, device=dev) + (w - 1) * (seq + 1)
    line = torch.empty(total + n * (w - 1), case["channels"], device=dev, dtype=kind)
    line[own_at] = rows
    back = torch.arange(w - 1, device=dev)
    line[first[:, None] + back] = s["tails"][ids, 0]
    o = s["bias"].float().expand(total, -1) if s["bias"] is not None else torch.zeros(1, device=dev)
    for j in range(w):
        o = o + line[own_at - (w - 1) + j].float() * s["w"][:, j].float()
    o = (o * torch.sigmoid(o)).to(kind)
    if case["op"] == "multi":
        ends = first[:, None] + 1 + torch.arange(case["tokens"], device=dev)
        s["snaps"][s["snap_ids"].long(), 0] = line[ends[..., None] + back]
        o = o.unflatten(0, (n, case["tokens"]))
    s["tails"][ids, 0] = line[(first + lens)[:, None] + back]
    got = {"o": o, "tails": s["tails"]}
    if case["op"] == "multi":
        got["snapshots"] = s["snaps"]
    return got


def _plain_norm(s):
    case = s["case"]
    groups, size = case["groups"], case["size"]
    x, z, w = s["x"].float().unflatten(1, (groups, size)), s["z"].float().unflatten(1, (groups, size)), s["w"].float().view(groups, size)
    gate = z * torch.sigmoid(z)
    if case["first"]:
        x = x * gate
    o = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if not case["first"]:
        o = o * gate
    return {"o": o.flatten(1).to(_TYPES[case["out"]])}


def run(s):
    case = s["case"]
    kind, op = case["kind"], case["op"]
    if not own:
        if kind == "scan":
            return _scan_prefill(s) if op == "prefill" else _scan_tokens(s)
        return _plain_conv(s) if kind == "conv" else _plain_norm(s)
    if kind == "norm":
        from rwkv_wkv_gb300 import gated_norm
        return {"o": gated_norm(s["x"], s["z"], s["w"], group_size=case["size"], eps=EPS, gate_first=case["first"],
                                out_dtype=_TYPES[case["out"]])}
    pool = s["pool"]
    if kind == "conv":
        if op == "decode":
            return {"o": pool.conv_step(0, s["ids"], s["u"], s["w"], s["bias"]), "tails": s["tails"]}
        if op == "multi":
            o = pool.conv_multi(0, s["ids"], s["u"], s["w"], s["bias"], step_snap_ids=s["snap_ids"])
            return {"o": o, "tails": s["tails"], "snapshots": s["snaps"]}
        return {"o": pool.conv_prefill(0, s["ids"], s["cu"], s["u"], s["w"], s["bias"]), "tails": s["tails"]}
    x = (s["x"], s["dt"], s["A"], s["b"], s["c"])
    more = {"D": s["D"], "dt_bias": s["bias"], "dt_softplus": True}
    if op == "decode":
        return {"o": pool.decode_step(0, s["ids"], *x, **more), "states": s["states"]}
    if op == "multi":
        o = pool.decode_multi(0, s["ids"], *x, step_snap_ids=s["snap_ids"], **more)
        return {"o": o, "states": s["states"], "snapshots": s["snaps"]}
    return {"o": pool.prefill(0, s["ids"], s["cu"], *x, max_seqlen=s["longest"], **more), "states": s["states"]}


# --------------------------------------------------------------------- in 64 bits

def _where(case, s):
    """For each token position: the rows at it, and which requests they belong to."""
    dev = s["ids"].device
    if case["op"] != "prefill":
        first = torch.arange(case["n"], device=dev) * case["tokens"]
        return [(first + t, slice(None)) for t in range(case["tokens"])]
    lens, first = lengths(case), s["cu"][:-1].long()
    if not case["ragged"]:
        return [(first + t, slice(None)) for t in range(lens[0])]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    by_length = torch.tensor(order, device=dev)
    alive, found = len(order), []
    for t in range(max(lens)):
        while lens[order[alive - 1]] <= t:
            alive -= 1
        some = by_length[:alive]
        found.append((first[some] + t, some))
    return found


def _exact_scan(case, s):
    h, share, ids = case["heads"], case["heads"] // case["groups"], s["ids"].long()
    rows = {k: s[k].flatten(0, 1) if case["op"] == "multi" else s[k] for k in ("x", "b", "c", "dt")}
    S = s["states"][ids, 0].double()
    A, D, bias = s["A"].double(), s["D"].double(), s["bias"].double()
    out = torch.zeros(rows["x"].shape, dtype=torch.float64, device=S.device)
    kept = s["snaps"].double() if "snaps" in s else None
    for t, (row, some) in enumerate(_where(case, s)):
        x = rows["x"][row].double()
        b, c = (rows[k][row].double().unsqueeze(2).expand(-1, -1, share, -1).flatten(1, 2) for k in "bc")
        dt = torch.logaddexp(rows["dt"][row].double() + bias, torch.zeros_like(bias))
        X = torch.exp(dt * A)[:, :, None, None] * S[some] + torch.einsum("bh,bhi,bhj->bhij", dt, x, b)
        out[row] = torch.einsum("bhij,bhj->bhi", X, c) + D[:, None] * x
        if kept is not None:
            X = X.to(s["snaps"].dtype).double() if case["state"] == "bf16" else X
            kept[s["snap_ids"][:, t].long(), 0] = X
        S[some] = X
    states = s["states"].double()
    states[ids, 0] = S
    got = {"o": out.unflatten(0, (case["n"], case["tokens"])) if case["op"] == "multi" else out, "states": states}
    if kept is not None:
        got["snapshots"] = kept
    return got


def _exact_conv(case, s):
    """Token after token, each request's window moved along by one."""
    ids = s["ids"].long()
    rows = s["u"].flatten(0, 1) if case["op"] == "multi" else s["u"]
    window = s["tails"][ids, 0].double()
    taps = s["w"].double().t()
    out = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
    kept = s["snaps"].double() if "snaps" in s else None
    for t, (row, some) in enumerate(_where(case, s)):
        full = torch.cat([window[some], rows[row].double()[:, None]], 1)
        y = torch.einsum("bjc,jc->bc", full, taps)
        if s["bias"] is not None:
            y += s["bias"].double()
        out[row] = y / (1 + torch.exp(-y))
        window[some] = full[:, 1:]
        if kept is not None:
            kept[s["snap_ids"][:, t].long(), 0] = full[:, 1:]
    tails = s["tails"].double()
    tails[ids, 0] = window
    got = {"o": out.unflatten(0, (case["n"], case["tokens"])) if case["op"] == "multi" else out, "tails": tails}
    if kept is not None:
        got["snapshots"] = kept
    return got


def _exact_norm(case, s):
    x, z, w = (s[k].double().view(-1, case["groups"], case["size"]) if k == "w" else
               s[k].double().reshape(case["rows"], case["groups"], case["size"]) for k in "xzw")
    gate = z / (1 + torch.exp(-z))
    u = x * gate if case["first"] else x
    o = w * u / torch.sqrt(u.square().sum(-1, keepdim=True) / case["size"] + EPS)
    return {"o": (o if case["first"] else o * gate).reshape(case["rows"], -1)}


def exact(case, seed):
    """The recurrences themselves in float64, token after token (the requests side by side), and the
    norm by its formula."""
    case = dict(case)
    s = _INPUTS[case["kind"]](case, seed)
    return {"scan": _exact_scan, "conv": _exact_conv, "norm": _exact_norm}[case["kind"]](case, s)
