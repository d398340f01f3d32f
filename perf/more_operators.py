"""The gated scan and linear cross attention as cases to be timed.

Gated scan: a recurrence with a gate of its own for every token and channel,

    h_t = a_t h_{t-1} + b_t,   y_t = h_t

``gate`` "decay": a = g, b = x;  "log": a = exp(g), b = x;  "sigmoid": a = sigmoid(g), b = (1 - a) x.
``scan`` runs a whole prompt (states in and out), ``scan_step`` one token for every row of a batch,
``scan_train`` the forward and the gradients of x, g and the start.

Linear cross attention: the keys and values of an encoder's tokens, of another number than the queries,

    S = sum_j phi(k_j) v_j^T,   z = sum_j phi(k_j),   y_t = phi(q_t) S / (phi(q_t) . z + eps)

(without the normaliser: y_t = phi(q_t) S).  ``cross`` sums up an encoder and reads it by a prompt's
queries, ``cross_step`` reads kept sums by one query for each row, ``cross_train`` is ``cross`` with the
gradients of q, k and v.  H query heads share Hk heads of keys and values.

A case's keys.  Scan: ``B`` sequences of ``N`` tokens, or packed ones of ``total`` tokens in all, the longest
``N``; ``D`` channels; ``carry``: from given states.  Cross: ``B`` sequences, ``Nq`` queries and ``N``
encoder tokens (padded: up to so many, from none on), packed where ``total`` and ``total_q`` say so.
"""

import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def _scan_case(op, B, N, D, dtype, gate, total=0, carry=True, name=None):
    c = dict(op=op, B=B, N=N, D=D, dtype=dtype, gate=gate, total=total, carry=carry)
    return dict(c, name=name) if name else c


def _cross_case(op, B, H, Hk, Nq, N, d, dtype, feature, layout, total_q=0, total=0, name=None):
    c = dict(op=op, B=B, H=H, Hk=Hk, Nq=Nq, N=N, d=d, dtype=dtype, feature=feature, layout=layout, total_q=total_q,
             total=total)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a chat turn of a single user: latency
        _scan_case("scan", 1, 77, 1024, "bf16", "sigmoid", name="scan_short"),
        # one very long document: the work has to be split along the sequence
        _scan_case("scan", 1, 65536, 1024, "bf16", "log", name="scan_long"),
        # one token of a small server batch: latency
        _scan_case("scan_step", 3, 1, 1024, "bf16", "sigmoid", name="scan_step_small"),
        # one token of a large one, wide channels, rows of a larger pool of states
        _scan_case("scan_step", 256, 1, 8192, "bf16", "sigmoid", name="scan_step_batch"),
        # an ordinary training batch: the benchmark's long sequences, 4 x 8192 tokens of 16 x 64 channels
        _scan_case("scan_train", 4, 8192, 1024, "bf16", "sigmoid", carry=False, name="scan_train_batch"),
        # documents of odd lengths packed into one row, full precision, carried from the rows before
        _scan_case("scan_train", 24, 4001, 384, "f32", "decay", total=20011, name="scan_train_packed"),
        # image tokens that read a prompt's 77 text tokens, padded, some prompts empty (no condition)
        _cross_case("cross", 8, 6, 6, 4096, 77, 64, "bf16", "elu1", "bnhd", name="cross_text"),
        # a short answer about one very long document, shared key heads
        _cross_case("cross", 1, 16, 4, 777, 65536, 128, "bf16", "elu1", "bnhd", name="cross_long"),
        # one token of a small server batch: latency
        _cross_case("cross_step", 3, 16, 16, 1, 1, 64, "bf16", "elu1", "bnhd", name="cross_step_small"),
        # the benchmark's decode batch, 256 x 16 heads, rows of a larger pool
        _cross_case("cross_step", 256, 16, 16, 1, 1, 64, "bf16", "elu1", "bnhd", name="cross_step_batch"),
        # training pairs, 4096 queries on up to 2048 encoder tokens
        _cross_case("cross_train", 8, 6, 6, 4096, 2048, 64, "bf16", "elu1", "qkv", name="cross_train_batch"),
        # packed pairs of odd lengths in full precision
        _cross_case("cross_train", 6, 6, 6, 1000, 700, 64, "f32", "elu1", "bhnd", total_q=2003, total=1501,
                    name="cross_train_f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _packed(rng, tokens, most):
    """(B, longest, total) of packed sequences of about ``tokens`` tokens, none longer than ``most``."""
    B = _log(rng, 1, min(24, tokens))
    total = min(tokens, most * B)
    longest = max(-(-total // B), min(most, total - B + 1, _log(rng, 1, most)))
    return B, longest, total


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_step", "scan_train", "scan_train", "cross", "cross", "cross_step",
                     "cross_train", "cross_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("scan"):
        gate = rng.choice(["sigmoid", "sigmoid", "log", "decay"])
        D = 8 * _log(rng, 2, 256)
        if op == "scan_step":
            return _scan_case(op, _log(rng, 1, 256), 1, 4 * D, dtype, gate)
        most = 1 << 25 if op == "scan" else 1 << 23
        tokens = _log(rng, 1, max(2, min(65536, most // D)))
        carry = rng.random() < 0.6
        if rng.random() < 0.4:
            B, longest, total = _packed(rng, tokens, 8192)
            return _scan_case(op, B, longest, D, dtype, gate, total=total, carry=carry)
        B = _log(rng, 1, min(16, tokens))
        return _scan_case(op, B, max(1, tokens // B), D, dtype, gate, carry=carry)
    d = rng.choice([16, 32, 64, 64, 128, 128])
    Hk = rng.choice([1, 2, 4, 6, 16])
    H = Hk * rng.choice([1, 1, 2, 4]) if Hk <= 4 else Hk
    feature = rng.choice(["elu1", "elu1", "exp", "identity"] + (["relu"] if op != "cross_train" else []))
    layout = rng.choice(["bhnd", "bnhd", "qkv"])
    if op == "cross_step":
        return _cross_case(op, _log(rng, 1, 256), H, Hk, 1, 1, d, dtype, feature, layout)
    most = (1 << 22 if op == "cross" else 1 << 20) // (4 if dtype == "f32" else 1)
    nq, nk = _log(rng, 1, max(2, most // (H * d) * 4)), _log(rng, 1, max(2, most // (Hk * d) * 4))
    if rng.random() < 0.4:
        B = _log(rng, 1, min(24, nq, nk))
        long_q = max(-(-nq // B), min(nq - B + 1, _log(rng, 1, 4096)))
        long_k = max(-(-nk // B), min(nk - B + 1, _log(rng, 1, 4096)))
        return _cross_case(op, B, H, Hk, long_q, long_k, d, dtype, feature, layout, total_q=nq, total=nk)
    B = _log(rng, 1, min(32, nq, nk))
    return _cross_case(op, B, H, Hk, max(1, nq // B), max(1, nk // B), d, dtype, feature, layout)


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _lengths(B, N, total, seed):
    """Lengths of B packed sequences: 1 .. N, one of them N or as near as it goes, together ``total``."""
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
    return share[torch.randperm(B, generator=g)]


def _offsets(B, N, total, seed):
    return torch.nn.functional.pad(torch.cumsum(_lengths(B, N, total, seed), 0), (1, 0)).int().cuda()


def _heads(case, g, b, n, heads, names, layout):
    """The named tensors, [b, heads, n, d] views of storage in the layout."""
    d, dt = case["d"], _dtype(case)
    if layout == "qkv" and len(names) > 1:
        x = torch.randn(b, n, len(names), heads, d, generator=g, device="cuda").to(dt)
        return {m: x[:, :, i].transpose(1, 2) for i, m in enumerate(names)}
    if layout == "bhnd":
        return {m: torch.randn(b, heads, n, d, generator=g, device="cuda").to(dt) for m in names}
    return {m: torch.randn(b, n, heads, d, generator=g, device="cuda").to(dt).transpose(1, 2) for m in names}


def _like(x):
    """An output beside x: token-major storage where x's is."""
    b, H, n, d = x.shape
    if x.stride(1) < x.stride(2):
        return torch.zeros(b, n, H, d, dtype=x.dtype, device=x.device).transpose(1, 2)
    return torch.zeros(b, H, n, d, dtype=x.dtype, device=x.device)


def _gates(case, g, shape):
    """Gates as a trained layer has them: channels that keep a few tokens to some thousands, varying by token."""
    D = case["D"]
    keep = 2 + 8 * (torch.arange(D, device="cuda") / max(D - 1, 1))  # 2^keep tokens, by channel
    n = torch.randn(*shape, generator=g, device="cuda")
    logit = (keep * math.log(2)).float() + n
    if case["gate"] == "sigmoid":
        return logit.to(_dtype(case))
    if case["gate"] == "log":
        return (-torch.exp(-logit)).to(_dtype(case))
    return torch.exp(-torch.exp(-logit)).to(_dtype(case))


def _prepare_scan(case, seed):
    g = _gen(seed)
    B, N, D, dt = case["B"], case["N"], case["D"], _dtype(case)
    step = case["op"] == "scan_step"
    shape = (B, D) if step else (1, case["total"], D) if case["total"] else (B, N, D)
    st = {"case": case, "g": _gates(case, g, shape)}
    st["x"] = torch.randn(*shape, generator=g, device="cuda").to(dt)
    st["y"] = torch.zeros(shape, dtype=dt, device="cuda")
    st["cu"] = _offsets(B, N, case["total"], seed) if case["total"] else None
    if case["op"] == "scan_train":
        st["dy"] = torch.randn(*shape, generator=g, device="cuda").to(dt)
        st["dx"], st["dg"] = torch.zeros_like(st["x"]), torch.zeros_like(st["g"])
        if case["carry"]:
            st["h0"] = torch.randn(B, D, generator=g, device="cuda")
            st["dh_last"] = torch.randn(B, D, generator=g, device="cuda")
            st["dh0"] = torch.zeros(B, D, device="cuda")
        return st
    slots = B + B // 4 + 1
    st["states"] = torch.randn(slots, D, generator=g, device="cuda")
    st["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].int()
    return st


def _prepare_cross(case, seed):
    g = _gen(seed)
    B, H, Hk, Nq, N, d = (case[n] for n in ("B", "H", "Hk", "Nq", "N", "d"))
    st = {"case": case}
    if case["op"] == "cross_step":
        slots = B + B // 4 + 1
        st["q"] = _heads(case, g, B, 1, H, "q", case["layout"])["q"]
        st["S"] = torch.randn(slots, Hk, d, d, generator=g, device="cuda") * 8
        st["z"] = torch.rand(slots, Hk, d, generator=g, device="cuda") * 64 + 32
        st["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].int()
        st["y"] = torch.zeros_like(st["q"])
        return st
    packed = case["total"] > 0
    layout = case["layout"]
    st.update(_heads(case, g, *((1, case["total_q"]) if packed else (B, Nq)), H, "q", layout))
    st.update(_heads(case, g, *((1, case["total"]) if packed else (B, N)), Hk, "kv", layout))
    st["cu_q"] = _offsets(B, Nq, case["total_q"], seed) if packed else None
    st["cu_k"] = _offsets(B, N, case["total"], seed + 1) if packed else None
    if not packed:  # padded encoder rows: most of them full or nearly so, one in eight empty
        st["lens"] = (N - (torch.rand(B, generator=g, device="cuda") ** 3 * N).floor()).int()
        st["lens"][7::8] = 0
    st["y"] = _like(st["q"])
    st["S"] = torch.zeros(B, Hk, d, d, device="cuda")
    st["z"] = torch.zeros(B, Hk, d, device="cuda")
    if case["op"] == "cross_train":
        st["dy"] = torch.randn(st["q"].shape, generator=g, device="cuda").to(st["q"].dtype)
        st.update({"d" + n: _like(st[n]) for n in "qkv"})
    return st


def prepare(case, seed):
    return _prepare_scan(case, seed) if case["op"].startswith("scan") else _prepare_cross(case, seed)


# ------------------------------------------------------------------------------ plain form: scan
def _gate(g, x, gate):
    """a and b of the recurrence, and the factor of x in b (None: 1), in 32 bits."""
    if gate == "decay":
        return g, x, None
    if gate == "log":
        return torch.exp(g), x, None
    rest = torch.sigmoid(-g)
    return torch.sigmoid(g), rest * x, rest


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero: pairs of tokens first, then the scan of the pairs."""
    n = a.shape[1]
    if n == 1:
        return b
    if n % 2:
        a, b = (torch.nn.functional.pad(t, (0, 0, 0, 1)) for t in (a, b))
    a0, a1, b0, b1 = a[:, 0::2], a[:, 1::2], b[:, 0::2], b[:, 1::2]
    odd = _scan(a1 * a0, a1 * b0 + b1)
    even = b0 + a0 * torch.nn.functional.pad(odd, (0, 0, 1, 0))[:, :-1]
    return torch.stack((even, odd), 2).flatten(1, 2)[:, :n]


def _firsts(st):
    """Rows (batch, token) of the sequences' first and last tokens."""
    case = st["case"]
    if st["cu"] is not None:
        cu = st["cu"].long()
        return torch.zeros_like(cu[:-1]), cu[:-1], cu[1:] - 1
    b = torch.arange(case["B"], device="cuda")
    return b, torch.zeros_like(b), torch.full_like(b, case["N"] - 1)


def _scan_parts(st, h0):
    """a (zero where a sequence starts), the full a, h, h_{t-1}, the factor of x, x and g in 32 bits."""
    g, x = st["g"].float(), st["x"].float()
    full, b, rest = _gate(g, x, st["case"]["gate"])
    rb, first, last = _firsts(st)
    a = full.clone()
    a[rb, first] = 0
    if h0 is not None:
        b = b.clone()
        b[rb, first] += full[rb, first] * h0
    h = _scan(a, b)
    return a, full, h, rest, x


def _plain_scan(st):
    case = st["case"]
    if case["op"] == "scan_step":
        at = st["slots"].long()
        a, b, _ = _gate(st["g"].float(), st["x"].float(), case["gate"])
        h = a * st["states"][at] + b
        st["states"][at] = h
        return h.to(st["y"].dtype), st["states"]
    rb, first, last = _firsts(st)
    if case["op"] == "scan":
        at = st["slots"].long()
        _, _, h, _, _ = _scan_parts(st, st["states"][at] if case["carry"] else None)
        st["states"][at] = h[rb, last]
        return h.to(st["y"].dtype), st["states"]
    h0 = st.get("h0")
    a, full, h, rest, x = _scan_parts(st, h0)
    before = torch.nn.functional.pad(h, (0, 0, 1, 0))[:, :-1].clone()
    before[rb, first] = 0 if h0 is None else h0
    dy = st["dy"].float().clone()
    if h0 is not None:
        dy[rb, last] += st["dh_last"]
    later = torch.nn.functional.pad(a, (0, 0, 0, 1))[:, 1:]
    G = _scan(later.flip(1), dy.flip(1)).flip(1)
    dt = st["x"].dtype
    if case["gate"] == "decay":
        dx, dg = G, G * before
    elif case["gate"] == "log":
        dx, dg = G, full * G * before
    else:
        dx, dg = rest * G, full * rest * G * (before - x)
    out = (h.to(dt), dx.to(dt), dg.to(dt))
    return out if h0 is None else (*out, (full * G)[rb, first])


# ----------------------------------------------------------------------------- plain form: cross
def _phi(x, feature):
    if feature == "elu1":
        return torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))
    return torch.exp(x) if feature == "exp" else x.clamp(min=0) if feature == "relu" else x


def _dphi(x, feature):
    if feature == "elu1":
        return torch.exp(x.clamp(max=0))
    return torch.exp(x) if feature == "exp" else (x > 0).float() if feature == "relu" else torch.ones_like(x)


def _live(case, st, which):
    """Indexes of the packed rows as a padded batch [B, n] (None: a padded batch already) and which are tokens."""
    n = case["Nq"] if which == "q" else case["N"]
    i = torch.arange(n, device="cuda")
    cu = st["cu_" + which]
    if cu is None:
        return None, (torch.ones(case["B"], n, dtype=torch.bool, device="cuda") if which == "q" else i < st["lens"][:, None])
    at = cu[:-1, None].long() + i
    return at.clamp(max=int(case["total_q" if which == "q" else "total"]) - 1), at < cu[1:, None]


def _wide(x, rows, live):
    """[B, H, n, d] in 32 bits, padded with zeros behind each sequence."""
    x = x.float() if rows is None else x[0][:, rows].transpose(0, 1).float()
    return torch.where(live[:, None, :, None], x, 0.0)


def _back(x, to, rows, live):
    """Writes the padded batch x into the rows of ``to``, rounded once; padding becomes zero."""
    if rows is None:
        to.copy_(torch.where(live[:, None, :, None], x, 0.0))
    else:
        to[0][:, rows[live]] = x.transpose(0, 1)[:, live].to(to.dtype)
    return to


def _groups(x, Hk):
    """[B, H, n, d] -> [B, Hk, H / Hk, n, d]."""
    return x.unflatten(1, (Hk, x.shape[1] // Hk))


def _read(fq, S, z, normalise):
    """Outputs and denominators (None without) of the features fq [B, Hk, G, n, d]."""
    num = fq @ S[:, :, None]
    if not normalise:
        return num, None
    den = (fq * z[:, :, None, None]).sum(-1, keepdim=True) + EPS
    return num / den, den


def _plain_cross(st):
    case = st["case"]
    f, Hk = case["feature"], case["Hk"]
    normalise = f != "identity"
    if case["op"] == "cross_step":
        at = st["slots"].long()
        fq = _groups(_phi(st["q"].float(), f), Hk)
        return _read(fq, st["S"][at], st["z"][at], normalise)[0].flatten(1, 2).to(st["q"].dtype)
    rows_q, live_q = _live(case, st, "q")
    rows_k, live_k = _live(case, st, "k")
    q, k, v = _wide(st["q"], rows_q, live_q), _wide(st["k"], rows_k, live_k), _wide(st["v"], rows_k, live_k)
    fq = _groups(_phi(q, f), Hk)
    fk = torch.where(live_k[:, None, :, None], _phi(k, f), 0.0)
    S, z = fk.transpose(-1, -2) @ v, fk.sum(2)
    y, den = _read(fq, S, z, normalise)
    y = _back(y.flatten(1, 2), st["y"], rows_q, live_q)
    if case["op"] == "cross":
        return y, S, z
    dy = _groups(_wide(st["dy"], rows_q, live_q), Hk)
    u = dy @ S.transpose(-1, -2)[:, :, None]
    if normalise:
        dden = -(fq * u).sum(-1, keepdim=True) / (den * den)
        dfq = u / den + dden * z[:, :, None, None]
        w = fq / den
        dz = (fq * dden).sum((2, 3))
    else:
        dfq, w, dz = u, fq, torch.zeros_like(z)
    w = torch.where(live_q[:, None, None, :, None], w, 0.0)
    dS = (w.transpose(-1, -2) @ dy).sum(2)
    dq = _dphi(q, f) * dfq.flatten(1, 2)
    dk = _dphi(k, f) * (v @ dS.transpose(-1, -2) + dz[:, :, None])
    dv = fk @ dS
    return (y, _back(dq, st["dq"], rows_q, live_q), _back(dk, st["dk"], rows_k, live_k),
            _back(dv, st["dv"], rows_k, live_k))


# --------------------------------------------------------------------------------- library's calls
def _own_scan(st):
    import token_level_head_gb300 as lib

    case = st["case"]
    kw = dict(gate=case["gate"])
    if case["op"] == "scan_step":
        lib.gated_scan_step(st["x"], st["g"], st["states"], st["y"], slots=st["slots"], **kw)
        return st["y"], st["states"]
    kw["cu_seqlens"] = st["cu"]
    if case["op"] == "scan":
        lib.gated_scan_forward(st["x"], st["g"], st["y"], states=st["states"], slots=st["slots"],
                               load_state=case["carry"], **kw)
        return st["y"], st["states"]
    if "checkpoints" not in st:  # a program allocates them once
        st["checkpoints"] = torch.empty(lib.gated_scan_checkpoint_rows(*st["x"].shape[:2]), case["D"], device="cuda")
    if not case["carry"]:
        lib.gated_scan_forward(st["x"], st["g"], st["y"], checkpoints=st["checkpoints"], **kw)
        lib.gated_scan_backward(st["x"], st["g"], st["dy"], st["checkpoints"], st["dx"], st["dg"], **kw)
        return st["y"], st["dx"], st["dg"]
    states = st["h0"].clone()  # the backward pass needs the start again
    lib.gated_scan_forward(st["x"], st["g"], st["y"], states=states, load_state=True, checkpoints=st["checkpoints"], **kw)
    lib.gated_scan_backward(st["x"], st["g"], st["dy"], st["checkpoints"], st["dx"], st["dg"], h0=st["h0"],
                            dh_last=st["dh_last"], dh0=st["dh0"], **kw)
    return st["y"], st["dx"], st["dg"], st["dh0"]


def _own_cross(st):
    import token_level_head_gb300 as lib

    case = st["case"]
    kw = dict(feature=case["feature"], normalise=case["feature"] != "identity")
    if "workspace" not in st:  # a program allocates it once
        size = lib.linattn_cross_workspace_bytes(case["B"], case["H"], case["Hk"], case["total_q"] or case["B"] * case["Nq"],
                                                 case["total"] or case["B"] * case["N"], case["d"],
                                                 backward=case["op"] == "cross_train")
        st["workspace"] = lib.new_workspace(size, st["q"].device)
    kw["workspace"] = st["workspace"]
    if case["op"] == "cross_step":
        return lib.linattn_cross_read(st["q"], st["S"], st["z"], st["y"], slots=st["slots"], eps=EPS, **kw)
    lens = st.get("lens")
    lib.linattn_cross_states(st["k"], st["v"], st["S"], st["z"], cu_seqlens=st["cu_k"], lens=lens, **kw)
    lib.linattn_cross_read(st["q"], st["S"], st["z"], st["y"], cu_seqlens=st["cu_q"], eps=EPS, **kw)
    if case["op"] == "cross":
        return st["y"], st["S"], st["z"]
    lib.linattn_cross_backward(st["q"], st["k"], st["v"], st["S"], st["z"], st["dy"], st["dq"], st["dk"], st["dv"],
                               cu_seqlens_q=st["cu_q"], cu_seqlens_k=st["cu_k"], lens=lens, eps=EPS, **kw)
    return st["y"], st["dq"], st["dk"], st["dv"]


def run(state):
    scan = state["case"]["op"].startswith("scan")
    if own:
        return _own_scan(state) if scan else _own_cross(state)
    return _plain_scan(state) if scan else _plain_cross(state)


# -------------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, op = case["B"], case["op"]
    if op.startswith("scan"):
        D, tokens = case["D"], case["total"] or B * case["N"]
        ops = 2 + (0 if case["gate"] == "decay" else 1 if case["gate"] == "log" else 4)
        state = B * D * 4
        if op == "scan_train":  # x, g in, y out; x, g, dy in, dx, dg out; the start twice, its gradient and the end's
            return {"bytes": 8 * tokens * D * es + (4 * state if case["carry"] else 0), "flops": (2 * ops + 7) * tokens * D}
        return {"bytes": 3 * tokens * D * es + (2 if case["carry"] else 1) * state, "flops": ops * tokens * D}
    H, Hk, d = case["H"], case["Hk"], case["d"]
    state = B * Hk * (d * d + d) * 4
    nq = (case["total_q"] or B * case["Nq"]) * H
    if op == "cross_step":
        return {"bytes": state + 2 * nq * d * es, "flops": 2 * nq * d * (d + 1)}
    nk = (case["total"] or B * case["N"]) * Hk
    forward, flops = (2 * nq + 2 * nk) * d * es, 2 * (nq + nk) * d * (d + 1)
    if op == "cross":
        return {"bytes": forward + state, "flops": flops}
    return {"bytes": forward + (3 * nq + 4 * nk) * d * es, "flops": flops + 4 * (nq + nk) * d * (d + 1)}


# ------------------------------------------------------------------------------------------- exact
def _exact_scan(case, seed):
    """Token by token in 64 bits."""
    st = _prepare_scan(case, seed)
    g, x = st["g"].double(), st["x"].double()
    keep = {"decay": lambda t: t, "log": torch.exp, "sigmoid": lambda t: 1 / (1 + torch.exp(-t))}[case["gate"]]
    a = keep(g)
    take = 1 / (1 + torch.exp(g)) if case["gate"] == "sigmoid" else torch.ones_like(g)
    b = take * x
    if case["op"] == "scan_step":
        states = st["states"].double()
        at = st["slots"].long()
        states[at] = a * states[at] + b
        return states[at], states
    cu = None if st["cu"] is None else st["cu"].tolist()
    spans = [(slice(None), 0, case["N"])] if cu is None else [(slice(0, 1), s, e) for s, e in zip(cu, cu[1:])]
    owner = [slice(None)] if cu is None else [slice(i, i + 1) for i in range(case["B"])]
    start = torch.zeros(case["B"], case["D"], dtype=torch.float64, device="cuda")
    if case["op"] == "scan" and case["carry"]:
        start = st["states"][st["slots"].long()].double()
    if "h0" in st:
        start = st["h0"].double()
    y, end = torch.zeros_like(x), start.clone()
    for (r, s, e), o in zip(spans, owner):
        h = start[o]
        for t in range(s, e):
            h = torch.addcmul(b[r, t], a[r, t], h)
            y[r, t] = h
        end[o] = h
    if case["op"] == "scan":
        states = st["states"].double()
        states[st["slots"].long()] = end
        return y, states
    dy, dx, dg = st["dy"].double(), torch.zeros_like(x), torch.zeros_like(x)
    dh0 = torch.zeros_like(start)
    for (r, s, e), o in zip(spans, owner):
        c = st["dh_last"].double()[o] if "dh_last" in st else torch.zeros_like(start[o])
        G = torch.zeros_like(x[r, s:e])
        for t in reversed(range(s, e)):
            G[:, t - s] = c = dy[r, t] + c
            c = a[r, t] * c
        dh0[o] = c
        last = torch.cat((start[o][:, None], y[r, s:e - 1]), 1)
        if case["gate"] == "sigmoid":
            last = (last - x[r, s:e]) * take[r, s:e]
        dg[r, s:e] = G * last * (1 if case["gate"] == "decay" else a[r, s:e])
        dx[r, s:e] = take[r, s:e] * G
    return (y, dx, dg, dh0) if "h0" in st else (y, dx, dg)


def _exact_cross(case, seed):
    """Sequence by sequence and head by head in 64 bits; the gradients through the weights' definition."""
    st = _prepare_cross(case, seed)
    f = case["feature"]
    feat = {"elu1": lambda x: torch.nn.functional.elu(x) + 1, "exp": torch.exp, "relu": torch.relu, "identity": lambda x: x}[f]
    slope = {"elu1": lambda x: torch.exp(torch.minimum(x, torch.zeros_like(x))), "exp": torch.exp,
             "relu": lambda x: (x > 0).double(), "identity": torch.ones_like}[f]
    B, H, Hk = case["B"], case["H"], case["Hk"]
    per, normalise = H // Hk, f != "identity"
    if case["op"] == "cross_step":
        at = st["slots"].long()
        S, z = (st[n][at].double().repeat_interleave(per, 1) for n in "Sz")
        x = feat(st["q"].double())
        y = torch.einsum("bhnc,bhce->bhne", x, S)
        return y / (torch.einsum("bhnc,bhc->bhn", x, z) + EPS)[..., None] if normalise else y
    q, k, v = (st[n].double() for n in "qkv")
    y, S, z = torch.zeros_like(q), st["S"].double(), st["z"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lens = st["lens"].tolist() if st["cu_k"] is None else None
    cq, ck = (None if st[n] is None else st[n].tolist() for n in ("cu_q", "cu_k"))
    for i in range(B):
        r, sq, sk = (i, slice(None), slice(0, lens[i])) if lens is not None else (0, slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1]))
        for h in range(Hk):
            fk, w = feat(k[r, h, sk]), v[r, h, sk]
            S[i, h], z[i, h] = fk.t() @ w, fk.sum(0)
            dS, dz = torch.zeros_like(S[i, h]), torch.zeros_like(z[i, h])
            for m in range(h * per, (h + 1) * per):
                fq = feat(q[r, m, sq])
                den = fq @ z[i, h] + EPS if normalise else torch.ones_like(fq[:, 0])
                out = (fq @ S[i, h]) / den[:, None]
                y[r, m, sq] = out
                if case["op"] == "cross":
                    continue
                dn = st["dy"][r, m, sq].double() / den[:, None]
                dd = -(dn * out).sum(1) * (1.0 if normalise else 0.0)
                dq[r, m, sq] = slope(q[r, m, sq]) * (dn @ S[i, h].t() + dd[:, None] * z[i, h])
                dS += fq.t() @ dn
                dz += fq.t() @ dd
            if case["op"] == "cross_train":
                dk[r, h, sk] = slope(k[r, h, sk]) * (w @ dS.t() + dz)
                dv[r, h, sk] = fk @ dS
    return (y, S, z) if case["op"] == "cross" else (y, dq, dk, dv)


def exact(case, seed):
    return _exact_scan(case, seed) if case["op"].startswith("scan") else _exact_cross(case, seed)
