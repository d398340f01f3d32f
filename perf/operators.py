"""The retention operators (linear attention with a decay for each head) as cases to be timed.

For a head with decay g, feature map phi and scale c, a sequence of tokens gives

    S_t = g S_{t-1} + phi(k_t) v_t^T,        y_t = c phi(q_t) S_t

Four operators work on it: ``prompt`` (a whole prompt in chunks, state in and out), ``step`` (one
token for every row of a batch), ``train`` (the gradients of q, k and v) and ``copy`` (states forked,
moved and cleared between the slots of a pool).  ``run`` takes the same state through the plain form
below or, with ``own``, through the library's calls.

A case's keys: ``op``; ``H`` heads of width ``d``; ``dtype`` of q, k, v ("bf16" or "f32"); ``feature``;
``layout`` of the token tensors ("bhnd": as they are, "bnhd": token-major, "qkv": slices of one
[.., 3, H, d] projection); ``B`` and ``N`` for a dense batch, or ``B`` sequences of ``total`` tokens
packed one behind another, the longest ``N``; ``carry``: the sequences start from the states of their slots.
"""

import math

import torch

own = False

CHUNK = 128


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a chat turn of a single user: latency
        dict(name="prompt_short", op="prompt", B=1, H=16, N=77, d=64, dtype="bf16", feature="identity",
             layout="qkv", total=0, carry=True),
        # the long causal sequences of the benchmark (4 x 16 heads x 8192), token-major as a projection writes them
        dict(name="prompt_batch", op="prompt", B=4, H=16, N=8192, d=64, dtype="bf16", feature="identity",
             layout="bnhd", total=0, carry=False),
        # one very long document with few heads: the work has to be split along the sequence
        dict(name="prompt_long", op="prompt", B=1, H=8, N=65536, d=128, dtype="bf16", feature="identity",
             layout="bnhd", total=0, carry=True),
        # a server's mixed batch of prompts, packed, lengths from one token on
        dict(name="prompt_packed", op="prompt", B=24, H=16, N=4001, d=128, dtype="bf16", feature="identity",
             layout="qkv", total=20011, carry=True),
        # full precision with the library's own feature map
        dict(name="prompt_f32", op="prompt", B=2, H=6, N=4096, d=64, dtype="f32", feature="elu1",
             layout="bhnd", total=0, carry=False),
        # one token of a small server batch: latency
        dict(name="step_small", op="step", B=3, H=16, N=1, d=128, dtype="bf16", feature="identity",
             layout="qkv", total=0, carry=True),
        # the benchmark's decode batch, 256 x 16 heads, rows of a larger pool of states
        dict(name="step_batch", op="step", B=256, H=16, N=1, d=64, dtype="bf16", feature="identity",
             layout="qkv", total=0, carry=True),
        # a short full-precision sample
        dict(name="train_f32", op="train", B=2, H=4, N=500, d=64, dtype="f32", feature="elu1",
             layout="bhnd", total=0, carry=False),
        # an ordinary training batch
        dict(name="train_batch", op="train", B=4, H=16, N=4096, d=64, dtype="bf16", feature="identity",
             layout="bnhd", total=0, carry=False),
        # documents of odd lengths packed into one row, wide heads
        dict(name="train_packed", op="train", B=12, H=16, N=4096, d=128, dtype="bf16", feature="identity",
             layout="bnhd", total=16384, carry=False),
        # one prompt's state forked to parallel samples, two slots cleared for new requests
        dict(name="copy_fork", op="copy", B=8, H=16, N=1, d=64, dtype="f32", feature="identity",
             layout="fork", total=0, carry=True),
        # a pool compacted after many requests have ended
        dict(name="copy_compact", op="copy", B=160, H=16, N=1, d=128, dtype="f32", feature="identity",
             layout="move", total=0, carry=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "train", "train", "copy"])
    d = rng.choice([16, 32, 64, 64, 128, 128])
    H = rng.choice([1, 3, 6, 8, 16, 20])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    feature = rng.choice(["identity", "identity", "elu1"])
    layout = rng.choice(["bhnd", "bnhd", "qkv"])
    if op == "copy":
        return dict(op=op, B=_log(rng, 1, 160), H=H, N=1, d=d, dtype="f32", feature="identity",
                    layout=rng.choice(["fork", "move"]), total=0, carry=True)
    if op == "step":
        return dict(op=op, B=_log(rng, 1, 256), H=H, N=1, d=d, dtype=dtype, feature=feature, layout=layout,
                    total=0, carry=True)
    # token-heads times width, at most the listed largest's
    most = {("prompt", "bf16"): 8 * 32768 * 128, ("prompt", "f32"): 12 * 4096 * 64,
            ("train", "bf16"): 64 * 2048 * 64, ("train", "f32"): 12 * 2048 * 64}[op, dtype]
    tokens = _log(rng, 1, max(2, most // (H * d)))
    carry = op == "prompt" and rng.random() < 0.5
    if rng.random() < 0.4:
        B = _log(rng, 1, 24)
        total = max(tokens, B)
        longest = max(-(-total // B), min(4096, total - B + 1, _log(rng, 1, 4096)))
        if total > B * longest or longest > 4096:
            total = min(total, 4096 * B)
            longest = min(4096, max(longest, -(-total // B)))
        return dict(op=op, B=B, H=H, N=longest, d=d, dtype=dtype, feature=feature, layout=layout, total=total,
                    carry=carry)
    B = _log(rng, 1, max(1, min(16, tokens)))
    return dict(op=op, B=B, H=H, N=max(1, tokens // B), d=d, dtype=dtype, feature=feature, layout=layout, total=0,
                carry=carry)


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _lengths(case, seed):
    """Lengths of the packed sequences: 1 .. N, one of them N, together ``total``."""
    B, N, total = case["B"], case["N"], case["total"]
    g = torch.Generator().manual_seed(int(seed) % (1 << 62) + 7)
    w = torch.exp(torch.rand(B, generator=g, dtype=torch.float64) * 5)
    first = min(N, total - (B - 1))
    w[0] = 0
    rest = total - first - (B - 1)
    share = (w / w.sum().clamp(min=1e-9) * max(rest, 0)).floor().long().clamp(max=N - 1) + 1
    share[0] = first
    short = torch.tensor(total) - share.sum()
    room = (N - share).clamp(min=0)
    before = torch.cumsum(room, 0) - room
    share = share + torch.minimum(room, (short - before).clamp(min=0))
    return share[torch.randperm(B, generator=g)].tolist()


def _tokens(case, g, lead, names, scale=1.0):
    """The named tensors, [.., H, N, d] views of storage in the case's layout."""
    H, d, dt = case["H"], case["d"], _dtype(case)
    b, n = lead
    if case["layout"] == "qkv":
        x = (torch.randn(b, n, len(names), H, d, generator=g, device="cuda") * scale).to(dt)
        return {m: x[:, :, i].transpose(1, 2) for i, m in enumerate(names)}
    if case["layout"] == "bnhd":
        return {m: (torch.randn(b, n, H, d, generator=g, device="cuda") * scale).to(dt).transpose(1, 2) for m in names}
    return {m: (torch.randn(b, H, n, d, generator=g, device="cuda") * scale).to(dt) for m in names}


def _like(x):
    """An output beside x: token-major storage where x's is."""
    b, H, n, d = x.shape
    if x.stride(1) < x.stride(2):
        return torch.zeros(b, n, H, d, dtype=x.dtype, device=x.device).transpose(1, 2)
    return torch.zeros(b, H, n, d, dtype=x.dtype, device=x.device)


def prepare(case, seed):
    g = _gen(seed)
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    h = torch.arange(H, dtype=torch.float64) / max(H - 1, 1)
    # the decays of multi-scale retention: 1 - 2^-5 for the first head to 1 - 2^-9 for the last
    st = {"case": case, "gamma": (1 - torch.exp2(-5 - 4 * h)).float().cuda(), "scale": d ** -0.5}
    if case["op"] == "copy":
        slots = B + B // 2 + 3
        st["states"] = torch.randn(slots, H, d, d, generator=g, device="cuda")
        perm = torch.randperm(slots, generator=torch.Generator().manual_seed(int(seed) % (1 << 62) + 3))
        if case["layout"] == "fork":
            src, dst = perm[:1].repeat(B), perm[1:1 + B].clone()
            src[-(B // 4):] = -1 if B >= 4 else src[-1]
        else:
            dst, src = torch.arange(B), perm[:B].clone()  # sources and targets overlap
            src[:: 16] = -1
        st["src"], st["dst"] = src.int().cuda(), dst.int().cuda()
        return st
    if case["op"] == "step":
        x = _tokens(case, g, (B, 1), "qkv")
        st.update({m: t[:, :, 0] for m, t in x.items()})
        slots = B + B // 4 + 1
        st["states"] = torch.randn(slots, H, d, d, generator=g, device="cuda")
        st["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].int()
        st["y"] = torch.zeros(B, H, d, dtype=_dtype(case), device="cuda")
        return st
    packed = case["total"] > 0
    lead = (1, case["total"]) if packed else (B, N)
    st.update(_tokens(case, g, lead, "qkv"))
    st["cu"] = None
    if packed:
        lens = torch.tensor([0] + _lengths(case, seed))
        st["cu"] = torch.cumsum(lens, 0).int().cuda()
    if case["op"] == "train":
        st["dy"] = _tokens(dict(case, layout="bnhd" if case["layout"] == "qkv" else case["layout"]), g, lead, ["dy"])["dy"]
        st.update({n: _like(st["q"]) for n in ("dq", "dk", "dv")})
        return st
    st["y"] = _like(st["q"])
    slots = B + 2
    st["states"] = torch.randn(slots, H, d, d, generator=g, device="cuda") if case["carry"] else \
        torch.zeros(slots, H, d, d, device="cuda")
    st["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].int()
    return st


# ------------------------------------------------------------------------------------- plain form
def _phi(x, feature):
    return torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0))) if feature == "elu1" else x


def _dphi(x, feature):
    return torch.exp(x.clamp(max=0)) if feature == "elu1" else torch.ones_like(x)


def _power(gamma, n):
    """gamma^n, [H, *n.shape], 0 where n < 0: 64-bit powers, for far positions, held in 32."""
    g = gamma.double().view(-1, *([1] * n.dim()))
    return torch.where(n >= 0, g ** n.clamp(min=0).double(), 0.0).float()


def _decayed(a, b, c, gamma, start=None):
    """sum_{s <= t} gamma^(t-s) (a_t . b_s) c_s + gamma^(t+1) a_t start, in chunks; [B, H, N, d], 32 bits."""
    B, H, N, d = a.shape
    n = -(-N // CHUNK)
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - N)).view(B, H, n, CHUNK, d) for x in (a, b, c))
    i = torch.arange(CHUNK, device=a.device)
    j = torch.arange(n, device=a.device)
    out = ((a @ b.transpose(-1, -2)) * _power(gamma, i[:, None] - i).unsqueeze(1)) @ c
    parts = (b * _power(gamma, CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ c
    state = (_power(gamma, CHUNK * (j[:, None] - 1 - j)) @ parts.view(B, H, n, d * d)).view(B, H, n, d, d)
    if start is not None:
        state = state + _power(gamma, CHUNK * j)[:, :, None, None] * start[:, :, None]
    out = out + _power(gamma, i + 1)[:, None, :, None] * (a @ state)
    return out.reshape(B, H, n * CHUNK, d)[:, :, :N]


def _rows(case, st):
    """Indexes of the packed rows as a padded batch [B, N] and which of them are tokens; None for a dense batch."""
    if st["cu"] is None:
        return None, None
    cu = st["cu"].long()
    at = cu[:-1, None] + torch.arange(case["N"], device=cu.device)
    return at.clamp(max=case["total"] - 1), at < cu[1:, None]


def _wide(x, rows, live):
    """[B, H, N, d] in 32 bits, padded with zeros behind each sequence."""
    x = x.float()
    if rows is None:
        return x
    return torch.where(live[:, None, :, None], x[0][:, rows].transpose(0, 1), 0.0)


def _back(x, to, rows, live):
    """Writes the padded batch x into the rows of ``to``, rounded once."""
    if rows is None:
        to.copy_(x)
    else:
        to[0][:, rows[live]] = x.transpose(0, 1)[:, live].to(to.dtype)
    return to


def _plain(st):
    case, gamma = st["case"], st["gamma"]
    f, scale = case["feature"], st["scale"]
    if case["op"] == "copy":
        src, dst = st["src"].long(), st["dst"].long()
        new = torch.where((src < 0)[:, None, None, None], 0.0, st["states"][src.clamp(min=0)])
        st["states"][dst] = new
        return st["states"]
    if case["op"] == "step":
        slots = st["slots"].long()
        q, k, v = (st[n].float() for n in "qkv")
        S = gamma[:, None, None] * st["states"][slots] + _phi(k, f)[..., :, None] * v[..., None, :]
        st["states"][slots] = S
        return (scale * (_phi(q, f)[..., None, :] @ S)[..., 0, :]).to(st["y"].dtype), st["states"]
    rows, live = _rows(case, st)
    q, k, v = (_wide(st[n], rows, live) for n in "qkv")
    fq, fk = _phi(q, f), _phi(k, f)
    if rows is not None:
        fq, fk = (torch.where(live[:, None, :, None], x, 0.0) for x in (fq, fk))
    if case["op"] == "train":
        dy = scale * _wide(st["dy"], rows, live)
        dq = _dphi(q, f) * _decayed(dy, v, fk, gamma)
        dk = _dphi(k, f) * _decayed(v.flip(2), dy.flip(2), fq.flip(2), gamma).flip(2)
        dv = _decayed(fk.flip(2), fq.flip(2), dy.flip(2), gamma).flip(2)
        return tuple(_back(x, st[n], rows, live) for x, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")))
    slots = st["slots"].long()
    S0 = st["states"][slots] if case["carry"] else None
    y = _back(scale * _decayed(fq, fk, v, gamma, S0), st["y"], rows, live)
    lens = live.sum(1) if rows is not None else torch.full((case["B"],), case["N"], device=q.device)
    left = lens[:, None] - 1 - torch.arange(case["N"], device=q.device)
    S = (fk * _power(gamma, left).transpose(0, 1)[..., None]).transpose(-1, -2) @ v
    if S0 is not None:
        S = S + _power(gamma, lens).t()[:, :, None, None] * S0
    st["states"][slots] = S
    return y, st["states"]


# --------------------------------------------------------------------------------- library's calls
def _own(st):
    import token_level_head_gb300 as lib

    case = st["case"]
    if case["op"] == "copy":
        return lib.retention_copy_states(st["states"], st["src"], st["dst"])
    kw = dict(scale=st["scale"], feature=case["feature"])
    if case["op"] == "step":
        lib.retention_step(st["q"], st["k"], st["v"], st["gamma"], st["states"], st["y"], slots=st["slots"], **kw)
        return st["y"], st["states"]
    if "workspace" not in st:  # a program allocates it once
        tokens = case["total"] or case["B"] * case["N"]
        size = lib.retention_workspace_bytes(case["B"], case["H"], tokens, case["d"], backward=case["op"] == "train")
        st["workspace"] = lib.new_workspace(size, st["q"].device)
    kw["workspace"] = st["workspace"]
    if st["cu"] is not None:
        kw["cu_seqlens"] = st["cu"]
    if case["op"] == "train":
        return lib.retention_backward(st["q"], st["k"], st["v"], st["gamma"], st["dy"], st["dq"], st["dk"], st["dv"], **kw)
    lib.retention_forward(st["q"], st["k"], st["v"], st["gamma"], st["y"], states=st["states"], slots=st["slots"],
                          load_state=case["carry"], **kw)
    return st["y"], st["states"]


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------------- work
def work(case):
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    slot = H * d * d * 4
    if case["op"] == "copy":
        cleared = B // 4 if case["layout"] == "fork" and B >= 4 else -(-B // 16) if case["layout"] == "move" else 0
        read = 1 if case["layout"] == "fork" else B - cleared
        return {"bytes": (read + B) * slot + 8 * B, "flops": 0}
    tokens = case["total"] or B * N
    if case["op"] == "step":
        return {"bytes": 2 * B * slot + 4 * B * H * d * es, "flops": 5 * B * H * d * d}
    if case["op"] == "train":  # q, k, v, dy in, dq, dk, dv out; both recurrences and three reads of a state
        return {"bytes": 7 * tokens * H * d * es, "flops": 10 * tokens * H * d * d}
    return {"bytes": 4 * tokens * H * d * es + (2 if case["carry"] else 1) * B * slot, "flops": 4 * tokens * H * d * d}


# ------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The recurrences token by token in 64 bits."""
    st = prepare(case, seed)
    g = st["gamma"].double()[None, :, None, None]
    if case["op"] == "copy":
        old = st["states"].double()
        new = old.clone()
        for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
            new[t] = old[s] if s >= 0 else 0
        return new
    elu = case["feature"] == "elu1"
    feat = (lambda x: torch.nn.functional.elu(x) + 1) if elu else (lambda x: x)
    slope = (lambda x: torch.exp(torch.minimum(x, torch.zeros_like(x)))) if elu else torch.ones_like
    scale = st["scale"]
    if case["op"] == "step":
        S = st["states"].double()
        at = st["slots"].long()
        q, k, v = (st[n].double() for n in "qkv")
        S[at] = g * S[at] + torch.einsum("bhc,bhe->bhce", feat(k), v)
        return scale * torch.einsum("bhc,bhce->bhe", feat(q), S[at]), S
    if case["total"]:
        cu = st["cu"].tolist()
        spans = [(0, cu[b], cu[b + 1]) for b in range(case["B"])]
    else:
        spans = [(b, 0, case["N"]) for b in range(case["B"])]
    # the sequences side by side, the longest first, so that those still running are a prefix
    order = sorted(range(len(spans)), key=lambda b: spans[b][1] - spans[b][2])
    spans = [spans[b] for b in order]
    lens = [e - s for _, s, e in spans]
    first = torch.tensor([s for _, s, _ in spans], device="cuda")
    batch = torch.tensor([b for b, _, _ in spans], device="cuda")
    alive = [sum(1 for n in lens if n > t) for t in range(lens[0])]
    x = {n: st[n].double() for n in ("q", "k", "v", "dy") if n in st}

    def at(name, t):
        m = alive[t]
        return x[name][batch[:m], :, first[:m] + t]

    def put(to, t, value):
        m = alive[t]
        to[batch[:m], :, first[:m] + t] = value

    S = torch.zeros(len(spans), case["H"], case["d"], case["d"], dtype=torch.float64, device="cuda")
    if case["op"] == "prompt":
        slots = st["slots"].long()[torch.tensor(order, device="cuda")]
        if case["carry"]:
            S.copy_(st["states"][slots])
        y = torch.zeros_like(x["q"])
        for t in range(lens[0]):
            m = alive[t]
            S[:m] = torch.baddbmm((g * S[:m]).flatten(0, 1), feat(at("k", t)).flatten(0, 1)[..., None],
                                  at("v", t).flatten(0, 1)[:, None]).view_as(S[:m])
            put(y, t, scale * (feat(at("q", t))[..., None, :] @ S[:m])[..., 0, :])
        states = st["states"].double()
        states[slots] = S
        return y, states
    dq, dk, dv = (torch.zeros_like(x["q"]) for _ in range(3))
    for t in range(lens[0]):
        m = alive[t]
        S[:m] = g * S[:m] + feat(at("k", t))[..., :, None] * at("v", t)[..., None, :]
        put(dq, t, slope(at("q", t)) * scale * (S[:m] @ at("dy", t)[..., None])[..., 0])
    G = torch.zeros_like(S)
    for t in reversed(range(lens[0])):
        m = alive[t]
        G[:m] = g * G[:m] + scale * feat(at("q", t))[..., :, None] * at("dy", t)[..., None, :]
        put(dk, t, slope(at("k", t)) * (G[:m] @ at("v", t)[..., None])[..., 0])
        put(dv, t, (feat(at("k", t))[..., None, :] @ G[:m])[..., 0, :])
    return dq, dk, dv
