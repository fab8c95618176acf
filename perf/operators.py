"""Cases, plain forms and 64-bit values of the gated delta rule and of draft verification.

Two operators of a server for models whose layers keep a recurrent state:

gated delta rule -- per value head a state S [head_v, head_k]; every token does
    S <- exp(g) S;  e = beta (v - S k);  S <- S + e k^T;  o = scale S q
  with q and k first divided by their length, sqrt(sum x^2 + eps).  Value head h reads
  query/key head h // (n_v_heads / n_k_heads).  It runs as one token for each of many
  slots ("decode"), as a few tokens for each of them with the state after every token
  kept ("multi", the pass that checks a draft), and over whole prompts ("prefill").

draft verification ("verify") -- rows of n_draft <= K drafted tokens.  Draft j is accepted
  while u_j q_j(d_j) < p_j(d_j); at the first refusal m the next token is the argmax of
  max(p_m - q_m, 0) / x over the vocabulary (x: exponential noise, so the argmax is a
  sample of the normalised residual; of p_m itself where the residual is empty, and of
  p_m / x after a fully accepted draft), the lowest index among equals.  It also names
  the stored state to go back to.

`run` computes the plain forms, or calls the library's GdnPool where `own` is set.
"""
import math
import random

import torch

own = False

EPS = 1e-6  # under the square root of the lengths of q and k


# ------------------------------------------------------------------------------ cases

def _gdn(op, name, heads, n, tokens=1, ragged=False, state="f32", inputs="bf16", out="bf16"):
    hk, hv, dk, dv = heads
    return {"name": name, "op": op, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "n": n, "tokens": tokens,
            "ragged": ragged, "state": state, "inputs": inputs, "out": out}


def _ver(name, n, k, vocab, pad=0, draft=True, ragged=False, probs="f32"):
    return {"name": name, "op": "verify", "n": n, "k": k, "vocab": vocab, "pad": pad, "draft": draft,
            "ragged": ragged, "probs": probs}


WIDE = (16, 32, 128, 128)   # two value heads for each query/key head


def listed():
    return [
        # one user's next token at one layer: latency
        _gdn("decode", "decode_one", WIDE, 1),
        # a full serving batch at one layer
        _gdn("decode", "decode_batch", WIDE, 256),
        # heads of 64, states kept in bf16, float32 inputs and outputs
        _gdn("decode", "decode_heads64", (12, 12, 64, 64), 201, state="bf16", inputs="f32", out="f32"),
        # the target model's pass over a draft of 4, with the five states to go back to
        _gdn("multi", "multi_check", WIDE, 48, tokens=5, out="f32"),
        # a short prompt that no tile divides
        _gdn("prefill", "prefill_short", WIDE, 1, tokens=77, out="f32"),
        # prompts of a mixed serving step: 64 sequences of 1 to 1,023 tokens
        _gdn("prefill", "prefill_ragged", WIDE, 64, tokens=512, ragged=True),
        # long prompts of a few users
        _gdn("prefill", "prefill_8x4096", WIDE, 8, tokens=4096),
        # one long document, few heads: little runs side by side
        _gdn("prefill", "prefill_long", (4, 8, 128, 128), 1, tokens=16383),
        # heads of 64 with states kept in bf16
        _gdn("prefill", "prefill_heads64", (32, 32, 64, 64), 8, tokens=1000, state="bf16"),
        # one user's draft of 4 over a 65,536-token vocabulary: latency
        _ver("verify_one", 1, 4, 65536),
        # a batch over a vocabulary whose rows are padded, drafts of differing lengths
        _ver("verify_batch", 256, 4, 130001, pad=79, ragged=True),
        # drafts copied from the prompt (no draft probabilities), bf16 rows of odd length
        _ver("verify_lookup", 64, 8, 65529, draft=False, probs="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_any(rng):
    op = rng.choice(("decode", "multi", "prefill", "prefill", "verify"))
    if op == "verify":
        draft = rng.random() < 0.7
        c = _ver("", _log_int(rng, 1, 256), rng.randint(1, 8), _log_int(rng, 1000, 140000), pad=rng.choice((0, 1, 8, 61)),
                 draft=draft, ragged=rng.random() < 0.5, probs=rng.choice(("f32", "f32", "bf16")))
    else:
        heads = rng.choice((WIDE, (4, 8, 128, 128), (2, 6, 128, 64), (3, 3, 64, 128), (12, 12, 64, 64), (32, 32, 64, 64)))
        kinds = dict(state=rng.choice(("f32", "f32", "bf16")), inputs=rng.choice(("bf16", "bf16", "f32")), out=rng.choice(("bf16", "f32")))
        if op == "decode":
            c = _gdn(op, "", heads, _log_int(rng, 1, 300), **kinds)
        elif op == "multi":
            kinds["state"] = "f32"
            c = _gdn(op, "", heads, _log_int(rng, 1, 64), tokens=rng.randint(2, 9), **kinds)
        else:
            kinds["inputs"] = "bf16"
            n = _log_int(rng, 1, 64)
            c = _gdn(op, "", heads, n, tokens=_log_int(rng, 1, max(2, 32768 // n // 2)), ragged=rng.random() < 0.5, **kinds)
    del c["name"]
    return c


def draw(rng):
    most = [work(c) for c in listed()]
    cap = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        c = _draw_any(rng)
        w = work(c)
        if w["bytes"] <= cap[0] and w["flops"] <= cap[1]:
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


def work(case):
    if case["op"] == "verify":
        n, e = case["n"], 2 if case["probs"] == "bf16" else 4
        # the target's row and the noise; the draft's row where a draft is refused (about half of the rows), and K values of each
        rows = e + 4 + (0.5 * e if case["draft"] else 0)
        return {"bytes": n * (case["vocab"] * rows + case["k"] * (2 * e + 12) + 8), "flops": 2.0 * n * case["vocab"]}
    rows, hv, dk, dv = _rows(case), case["hv"], case["dk"], case["dv"]
    ein = 2 if case["inputs"] == "bf16" else 4
    eout = 2 if case["out"] == "bf16" else 4
    est = 2 if case["state"] == "bf16" else 4
    per_row = (2 * case["hk"] * dk + hv * dv) * ein + 8 * hv + hv * dv * eout
    states = case["n"] * hv * dk * dv * est
    kept = rows * hv * dk * dv * est if case["op"] == "multi" else 0
    return {"bytes": float(rows * per_row + 2 * states + kept), "flops": 6.0 * rows * hv * dk * dv}


# ----------------------------------------------------------------------------- inputs

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(seed, dev):
    return torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)


def _gdn_inputs(case, seed):
    """The tokens as the layer's projections leave them: q, k and v beside each other in one buffer
    (after a SiLU), the log decay g = -A softplus(x + dt) <= 0 and the step beta in (0, 1)."""
    dev = _device()
    gen = _gen(seed, dev)
    hk, hv, dk, dv, n = case["hk"], case["hv"], case["dk"], case["dv"], case["n"]
    rows = _rows(case)
    wide = 2 * hk * dk + hv * dv
    x = torch.randn(rows, wide, device=dev, generator=gen)
    qkv = torch.nn.functional.silu(x).to(_TYPES[case["inputs"]])
    del x
    q = qkv[:, : hk * dk].unflatten(1, (hk, dk))
    k = qkv[:, hk * dk: 2 * hk * dk].unflatten(1, (hk, dk))
    v = qkv[:, 2 * hk * dk:].unflatten(1, (hv, dv))
    a = 1.0 + 15.0 * torch.rand(hv, device=dev, generator=gen)
    dt = torch.exp(torch.rand(hv, device=dev, generator=gen) * math.log(100.0) + math.log(1e-3))
    bias = dt + torch.log(-torch.expm1(-dt))          # softplus(bias) = dt
    g = -a * torch.nn.functional.softplus(torch.randn(rows, hv, device=dev, generator=gen) * 0.5 + bias)
    beta = torch.sigmoid(torch.randn(rows, hv, device=dev, generator=gen))
    slots = n + 3
    states = (torch.randn(slots, 1, hv, dv, dk, device=dev, generator=gen) * 0.1).to(_TYPES[case["state"]])
    ids = torch.randperm(slots, device=dev, generator=gen)[:n].to(torch.int32)
    s = {"case": case, "q": q, "k": k, "v": v, "g": g, "beta": beta, "ids": ids, "states": states}
    if case["op"] == "multi":
        t = case["tokens"]
        for name in ("q", "k", "v", "g", "beta"):
            s[name] = s[name].unflatten(0, (n, t))
        s["snaps"] = torch.zeros(n * t, 1, hv, dv, dk, device=dev, dtype=_TYPES[case["state"]])
        s["snap_ids"] = torch.randperm(n * t, device=dev, generator=gen).to(torch.int32).view(n, t)
    if case["op"] == "prefill":
        lens = torch.tensor(lengths(case), device=dev)
        s["cu"] = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
        s["longest"] = max(lengths(case))
    return s


def _verify_inputs(case, seed):
    """Softmax rows with a heavy head, a draft model that is near the target, drafts sampled from it."""
    dev = _device()
    gen = _gen(seed, dev)
    n, k, vocab = case["n"], case["k"], case["vocab"]
    ld, kind = vocab + case["pad"], _TYPES[case["probs"]]
    z = 2.5 * torch.randn(n, k + 1, vocab, device=dev, generator=gen)
    p = torch.zeros(n, k + 1, ld, device=dev, dtype=kind)[..., :vocab]
    p.copy_(torch.softmax(z, -1))
    q = None
    if case["draft"]:
        z = z[:, :k]
        z += 0.3 * torch.randn(n, k, vocab, device=dev, generator=gen)
        q = torch.zeros(n, k, ld, device=dev, dtype=kind)[..., :vocab]
        q.copy_(torch.softmax(z, -1))
        race = q.float() / torch.empty(n, k, vocab, device=dev).exponential_(generator=gen)
    else:  # drafts that the target finds likely
        race = p[:, :k].float() ** 1.5 / torch.empty(n, k, vocab, device=dev).exponential_(generator=gen)
    del z
    s = {"case": case, "p": p, "q": q, "ids": race.argmax(-1).to(torch.int32)}
    del race
    s["u"] = torch.rand(n, k, device=dev, generator=gen)
    s["noise"] = torch.zeros(n, ld, device=dev)[:, :vocab]
    s["noise"].copy_(torch.empty(n, vocab, device=dev).exponential_(generator=gen))
    s["n_draft"] = torch.randint(0, k + 1, (n,), device=dev, generator=gen, dtype=torch.int32) if case["ragged"] else None
    s["snap_ids"] = torch.randperm(n * (k + 1), device=dev, generator=gen).to(torch.int32).view(n, k + 1)
    return s


def prepare(case, seed):
    case = dict(case)
    if case["op"] == "verify":
        s = _verify_inputs(case, seed)
        if own:  # the handle that a server keeps: the pool whose stored states the row goes back to
            from rwkv_wkv_gb300 import GdnPool
            s["pool"] = GdnPool(1, 1, 1, 1, n_snapshots=case["n"] * (case["k"] + 1), head_k=64, head_v=64)
        return s
    s = _gdn_inputs(case, seed)
    if own:  # the same states, in the pool that a server keeps them in
        from rwkv_wkv_gb300 import GdnPool
        pool = GdnPool(1, case["hk"], case["hv"], len(s["states"]), n_snapshots=len(s["snaps"]) if "snaps" in s else 0,
                       head_k=case["dk"], head_v=case["dv"], state_dtype=case["state"], out_dtype=case["out"])
        pool.states.copy_(s["states"])
        s["pool"], s["states"] = pool, pool.states
        if "snaps" in s:
            pool.snapshots.zero_()
            s["snaps"] = pool.snapshots
    return s


# -------------------------------------------------------------------------- one pass

def _unit(x):
    x = x.float()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def _per_value_head(x, case):
    return x.repeat_interleave(case["hv"] // case["hk"], dim=-2)


def _step(state, q, k, v, g, beta, scale):
    """One token for each row: state [n, hv, dv, dk]; q, k [n, hv, dk]; v [n, hv, dv]; g, beta [n, hv]."""
    state = state * torch.exp(g)[..., None, None]
    e = beta[..., None] * (v - (state * k[..., None, :]).sum(-1))
    state = state + e[..., None] * k[..., None, :]
    return state, scale * (state * q[..., None, :]).sum(-1)


def _plain_decode(s):
    case = s["case"]
    q, k = (_per_value_head(_unit(s[x]), case) for x in "qk")
    at = s["ids"].long()
    state, o = _step(s["states"][at, 0].float(), q, k, s["v"].float(), s["g"], s["beta"], case["dk"] ** -0.5)
    s["states"][at, 0] = state.to(s["states"].dtype)
    return {"o": o.to(_TYPES[case["out"]]), "states": s["states"]}


def _plain_multi(s):
    case = s["case"]
    q, k = (_per_value_head(_unit(s[x]), case) for x in "qk")
    v, at = s["v"].float(), s["ids"].long()
    state = s["states"][at, 0].float()
    o = torch.empty(v.shape, device=v.device, dtype=_TYPES[case["out"]])
    for t in range(case["tokens"]):
        state, ot = _step(state, q[:, t], k[:, t], v[:, t], s["g"][:, t], s["beta"][:, t], case["dk"] ** -0.5)
        o[:, t] = ot.to(o.dtype)
        s["snaps"][s["snap_ids"][:, t].long(), 0] = state.to(s["snaps"].dtype)
    s["states"][at, 0] = state.to(s["states"].dtype)
    return {"o": o, "states": s["states"], "snapshots": s["snaps"]}


CHUNK = 64


def _plain_prefill(s):
    """By chunks of 64 tokens.  With G the running sum of g inside a chunk and D_ts = exp(G_t - G_s), the e_t of
    a chunk solve (I + A) E = diag(beta) (V - diag(exp G) K S^T), A_ts = beta_t D_ts <k_t, k_s> for s < t, and
        O = scale (diag(exp G) Q S^T + (Q K^T * D) E),   S <- exp(G_L) S + (diag(D_L) E)^T K."""
    case, dev = s["case"], s["q"].device
    n, hv, dk, dv = case["n"], case["hv"], case["dk"], case["dv"]
    chunks = max(1, -(-s["longest"] // CHUNK))
    lens = s["cu"].diff().long()
    pos = torch.arange(chunks * CHUNK, device=dev)
    live = pos[None] < lens[:, None]                                    # the padding is tokens that change nothing
    at = torch.where(live, s["cu"][:-1].long()[:, None] + pos[None], 0)

    def chunked(x, keep):  # [rows, heads, ...] -> [n, heads, chunks, 64, ...]
        x = x[at].float()
        x = torch.where(live.view(*live.shape, *([1] * (x.dim() - 2))), x, 0.0) if keep else x
        return x.transpose(1, 2).unflatten(2, (chunks, CHUNK))

    q = chunked(_per_value_head(_unit(s["q"]), case), False)
    k = chunked(_per_value_head(_unit(s["k"]), case), True)
    v = chunked(s["v"], False)
    beta, total = chunked(s["beta"], True), chunked(s["g"], True).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    decay = torch.where(low, total[..., :, None] - total[..., None, :], -math.inf).exp()
    a = (beta[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    inverse = torch.eye(CHUNK, device=dev).expand_as(a).clone()
    for i in range(1, CHUNK):  # forward substitution, a row of every chunk at a time
        inverse[..., i, :i] = -(a[..., i, None, :i] @ inverse[..., :i, :i])[..., 0, :]
    u = inverse @ (beta[..., None] * v)
    w = inverse @ ((beta * total.exp())[..., None] * k)
    p = decay * (q @ k.transpose(-1, -2))
    q = q * total.exp()[..., None]
    k = k * (total[..., -1:] - total).exp()[..., None]
    state = s["states"][s["ids"].long(), 0].float()
    o = torch.empty_like(v)
    for c in range(chunks):
        e = u[:, :, c] - w[:, :, c] @ state.transpose(-1, -2)
        o[:, :, c] = q[:, :, c] @ state.transpose(-1, -2) + p[:, :, c] @ e
        state = total[:, :, c, -1].exp()[..., None, None] * state + e.transpose(-1, -2) @ k[:, :, c]
    s["states"][s["ids"].long(), 0] = state.to(s["states"].dtype)
    return {"o": (dk ** -0.5 * o.flatten(2, 3).transpose(1, 2)[live]).to(_TYPES[case["out"]]), "states": s["states"]}


def _plain_verify(s):
    case = s["case"]
    k, rows = case["k"], torch.arange(case["n"], device=s["p"].device)
    d = s["ids"].long()
    drafted = s["n_draft"].long() if s["n_draft"] is not None else torch.full_like(rows, k)
    col = torch.arange(k + 1, device=d.device)
    pd = s["p"][:, :k].gather(-1, d[..., None])[..., 0].float()
    qd = s["q"].gather(-1, d[..., None])[..., 0].float() if s["q"] is not None else torch.ones_like(pd)
    taken = (s["u"] * qd < pd) & (col[:k] < drafted[:, None])
    m = taken.long().cumprod(1).sum(1)
    pm = s["p"][rows, m].float()
    refused = m < drafted
    last = m.clamp(max=k - 1)
    if s["q"] is not None:
        qm = torch.where(refused[:, None], s["q"][rows, last].float(), 0.0)
    else:
        qm = torch.zeros_like(pm)
        qm[rows, d[rows, last]] = refused.float()
    rest = (pm - qm).clamp(min=0)
    rest = torch.where((rest > 0).any(1, keepdim=True), rest, pm)
    token = torch.where(rest > 0, rest / s["noise"], -1.0).argmax(1)
    token = torch.where((rest > 0).any(1), token, -1)
    padded = torch.cat([d, d[:, :1]], 1)
    tokens = torch.where(col < m[:, None], padded, torch.where(col == m[:, None], token[:, None], -1))
    return {"accepted": m.to(torch.int32), "tokens": tokens.to(torch.int32), "resume": s["snap_ids"][rows, m]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"decode": _plain_decode, "multi": _plain_multi, "prefill": _plain_prefill, "verify": _plain_verify}[op](s)
    pool = s["pool"]
    if op == "verify":
        accepted, tokens, resume = pool.verify_drafts(s["ids"], s["p"], s["q"], s["u"], s["noise"],
                                                      n_draft=s["n_draft"], step_snap_ids=s["snap_ids"])
        return {"accepted": accepted, "tokens": tokens, "resume": resume}
    x = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if op == "decode":
        return {"o": pool.decode_step(0, s["ids"], *x, l2norm_eps=EPS), "states": s["states"]}
    if op == "multi":
        o = pool.decode_multi(0, s["ids"], *x, step_snap_ids=s["snap_ids"], l2norm_eps=EPS)
        return {"o": o, "states": s["states"], "snapshots": s["snaps"]}
    return {"o": pool.prefill(0, s["ids"], s["cu"], *x, max_seqlen=s["longest"], l2norm_eps=EPS), "states": s["states"]}


# --------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The recurrence itself, token after token in float64 (the sequences of a prefill side by side)."""
    if case["op"] == "verify":
        return None  # whole numbers
    s = _gdn_inputs(dict(case), seed)
    hv, dk = case["hv"], case["dk"]
    share = hv // case["hk"]
    ids = s["ids"].long()
    S = s["states"][ids, 0].double()
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=S.device)
    if case["op"] == "prefill":
        lens = lengths(case)
        first = s["cu"][:-1].long()
        steps = [(t, torch.tensor([i for i, x in enumerate(lens) if x > t], device=S.device)) for t in range(max(lens))] \
            if case["ragged"] else [(t, None) for t in range(max(lens))]
    else:
        flat = lambda x: x.flatten(0, 1) if case["op"] == "multi" else x  # noqa: E731
        for name in ("q", "k", "v", "g", "beta"):
            s[name] = flat(s[name])
        out = flat(out)
        first = torch.arange(case["n"], device=S.device) * case["tokens"]
        steps = [(t, None) for t in range(case["tokens"])]
    kept = s["snaps"].double() if "snaps" in s else None
    for t, some in steps:
        row = first + t if some is None else first[some] + t
        q, k = s["q"][row].double(), s["k"][row].double()
        q = (q / (q.square().sum(-1, keepdim=True) + EPS).sqrt() / math.sqrt(dk)).repeat_interleave(share, 1)
        k = (k / (k.square().sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(share, 1)
        X = (S if some is None else S[some]) * s["g"][row].double().exp()[:, :, None, None]
        e = s["beta"][row].double()[:, :, None] * (s["v"][row].double() - torch.einsum("bhij,bhj->bhi", X, k))
        X = X + torch.einsum("bhi,bhj->bhij", e, k)
        out[row] = torch.einsum("bhij,bhj->bhi", X, q)
        if some is None:
            S = X
        else:
            S[some] = X
        if kept is not None:
            kept[s["snap_ids"][:, t].long(), 0] = S
    states = s["states"].double()
    states[ids, 0] = S
    got = {"o": out.unflatten(0, (case["n"], case["tokens"])) if case["op"] == "multi" else out, "states": states}
    if kept is not None:
        got["snapshots"] = kept
    return got
