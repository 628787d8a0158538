"""The gated delta rule and the channel-last group norm: cases, plain forms and definitions.

Two operators stand next to the selective scan in a token mixer of this library, with their gradients:

* the gated delta rule, a linear recurrence with a matrix state per head,
      S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   a_t = exp(g_t),
      o_t = scale S_t^T q_t,
  over equal rows [B, L] or packed rows with offsets, its backward, and its single-token form on a pool of
  states (serving);
* the group norm of channel-last tokens [N, L, C] with an optional SiLU, and its backward.

`run` computes them in their plain form (torch, 32 bits) or, with `own`, by the library's entry points.
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_CHUNK = 64
_EPS_L2 = 1e-6
_EPS_GN = 1e-5


# ---------------------------------------------------------------- cases
def _gdr(name, op, B, L, Hk, H, dk, dv, io, **more):
    case = {"name": name, "op": op, "B": B, "L": L, "Hk": Hk, "H": H, "dk": dk, "dv": dv, "io": io,
            "l2norm": True, "h0": False, "state": False, "lens": 0}
    case.update(more)
    return case


def _gn(name, op, N, L, C, G, io, act="silu", affine=True):
    return {"name": name, "op": op, "N": N, "L": L, "C": C, "G": G, "io": io, "act": act, "affine": affine}


def listed():
    return [
        # the vision backbone's stage-4 rows (49 patches and two auxiliary tokens), 640 channels as 10 heads
        _gdr("gdr_fwd_stage4", "gdr_fwd", 256, 51, 10, 10, 64, 64, "bf16"),
        # its stage-3 rows, 320 channels as 5 heads, in 32 bits (a parity or small-batch run)
        _gdr("gdr_fwd_stage3_f32", "gdr_fwd", 32, 198, 5, 5, 64, 64, "f32"),
        # two long rows, wide heads, two value heads to a key head, the state handed on
        _gdr("gdr_fwd_long", "gdr_fwd", 2, 8192, 8, 16, 128, 128, "bf16", state=True),
        # ragged rows packed end to end (prefill of requests that go on from a state)
        _gdr("gdr_fwd_packed", "gdr_fwd", 24, 2048, 8, 8, 64, 128, "bf16", h0=True, state=True, lens=3),
        # training at stage 3
        _gdr("gdr_bwd_stage3", "gdr_bwd", 64, 198, 5, 5, 64, 64, "bf16"),
        # training on long rows with shared key heads
        _gdr("gdr_bwd_long", "gdr_bwd", 2, 4002, 4, 8, 128, 128, "bf16"),
        # one token of one stream: the smallest call, latency counts
        _gdr("gdr_step_one", "gdr_step", 1, 1, 5, 5, 64, 64, "f32"),
        # one token each of many requests, their states in a pool
        _gdr("gdr_step_batch", "gdr_step", 256, 1, 8, 16, 128, 128, "bf16"),
        # the mixer's output norm at stage 3: a group a head
        _gn("gn_fwd_stage3", "gn_fwd", 256, 198, 320, 5, "bf16"),
        # the stem's feature maps, 112 x 112, five channels to a group
        _gn("gn_fwd_image", "gn_fwd", 16, 12544, 160, 32, "bf16"),
        # training at stage 4
        _gn("gn_bwd_stage4", "gn_bwd", 256, 51, 640, 10, "bf16"),
        # training on feature maps in 32 bits
        _gn("gn_bwd_image_f32", "gn_bwd", 4, 12544, 320, 32, "f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_bwd", "gdr_step", "gn_fwd", "gn_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("gn"):
        G = rng.choice([1, 2, 4, 5, 8, 10, 16, 32])
        C = G * _log_int(rng, max(1, 32 // G), max(1, 1280 // G))
        L = _log_int(rng, 1, 16384)
        most = 16 * 12544 * 160 if io == "bf16" else 4 * 12544 * 320
        N = _log_int(rng, 1, max(1, min(4096, most // (L * C))))
        case = _gn("", op, N, L, C, G, io, rng.choice(["silu", "silu", "none"]), rng.random() < 0.8)
    else:
        Hk = rng.choice([1, 2, 4, 5, 8, 10])
        H = Hk * rng.choice([1, 1, 2, 4] if Hk < 8 else [1, 2])
        dk = rng.choice([16, 24, 32, 40, 64, 64, 80, 96, 128, 128])
        dv = rng.choice([dk, dk, 16, 32, 64, 100, 128, 192, 256])
        if op == "gdr_step":
            B = _log_int(rng, 1, max(1, 256 * 16 * 128 * 128 // (H * dk * dv)) if H * dk * dv > 16 * 128 * 128 else 256)
            case = _gdr("", op, B, 1, Hk, H, dk, dv, io)
        else:
            L = _log_int(rng, 1, 8192 if op == "gdr_fwd" else 4002)
            most = (2 * 8192 * 16 * 128 * 128 if op == "gdr_fwd" else 2 * 4002 * 8 * 128 * 128) // (4 if io == "f32" else 1)
            B = _log_int(rng, 1, max(1, min(512, most // (L * H * dk * max(dv, dk)))))
            h0 = rng.random() < 0.4
            case = _gdr("", op, B, L, Hk, H, dk, dv, io, h0=h0, state=op == "gdr_fwd" and (h0 or rng.random() < 0.3),
                        lens=rng.randint(1, 1000000) if rng.random() < 0.35 else 0)
        case["l2norm"] = rng.random() < 0.8
    del case["name"]
    return case


def _lengths(case):
    """The rows' lengths: all L, or (packed) spread over 1 .. L, some rows empty."""
    if not case["lens"]:
        return [case["L"]] * case["B"]
    r = random.Random(case["lens"])
    return [0 if r.random() < 0.05 else r.randint(1, case["L"]) for _ in range(case["B"])]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    io = _TYPES[case["io"]]
    normal = lambda *s: torch.randn(s, generator=gen, device=dev)
    uniform = lambda lo, hi, *s: lo + (hi - lo) * torch.rand(s, generator=gen, device=dev)
    st = {"case": case}
    if case["op"].startswith("gn"):
        N, L, C, G = case["N"], case["L"], case["C"], case["G"]
        # activations of a network: every channel has a mean and a scale of its own
        st["x"] = (normal(N, L, C) * uniform(0.3, 2.0, C) + normal(C)).to(io)
        st["w"] = uniform(0.5, 1.5, C) if case["affine"] else None
        st["b"] = 0.3 * normal(C) if case["affine"] else None
        if case["op"] == "gn_bwd":
            st["dy"] = normal(N, L, C).to(io)
            # what the forward pass left for the backward
            x = st["x"].float().view(N, L, G, C // G)
            st["mean"] = x.mean(dim=(1, 3))
            st["rstd"] = torch.rsqrt((x - st["mean"].view(N, 1, G, 1)).square().mean(dim=(1, 3)) + _EPS_GN)
        return st
    B, L, Hk, H, dk, dv = (case[n] for n in ("B", "L", "Hk", "H", "dk", "dv"))
    lens = _lengths(case)
    if case["op"] == "gdr_step":
        rows = (B,)
    elif case["lens"]:
        rows = (1, sum(lens))
    else:
        rows = (B, L)
    # queries and keys of a projection: neighbours in a row are alike; unit keys where the call does not norm them
    q, k = normal(*rows, Hk, dk), normal(*rows, Hk, dk) + 0.5 * normal(Hk, dk)
    if not case["l2norm"]:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    st["q"], st["k"], st["v"] = q.to(io), k.to(io), normal(*rows, H, dv).to(io)
    # log decays -A softplus(.): steps from 1e-3 to 1e-1, rates from 1 to 16; gates of a sigmoid
    st["g"] = -(uniform(0.0, math.log(16.0), H).exp() * uniform(math.log(1e-3), math.log(1e-1), *rows, H).exp()).to(io)
    st["beta"] = torch.sigmoid(normal(*rows, H)).to(io)
    if case["op"] == "gdr_step":
        pool = B + B // 4 + 1
        st["pool"] = normal(pool, H, dk, dv) / math.sqrt(dk)
        st["slots"] = torch.randperm(pool, generator=gen, device=dev)[:B].to(torch.int32)
        return st
    st["offsets"], st["max_len"] = None, L
    if case["lens"]:
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        st["offsets"], st["max_len"] = torch.tensor(ends, dtype=torch.int32, device=dev), max(lens + [1])
    st["h0"] = normal(B, H, dk, dv) / math.sqrt(dk) if case["h0"] else None
    if case["op"] == "gdr_bwd":
        st["do"] = normal(*rows, H, dv).to(io)
    return st


# ---------------------------------------------------------------- plain forms
def _padded(t, st, pad_to):
    """[B, L, ...] or packed [1, total, ...] -> float32 [B, pad_to, ...], zeros behind each row's end."""
    B = st["case"]["B"]
    if st["offsets"] is None:
        out = torch.zeros((B, pad_to) + t.shape[2:], device=t.device)
        out[:, :t.shape[1]] = t.float()
        return out
    at = st["offsets"][:-1, None].long() + torch.arange(pad_to, device=t.device)
    inside = at < st["offsets"][1:, None]
    flat = torch.cat([t[0].float(), torch.zeros((1,) + t.shape[2:], device=t.device)])
    return flat[torch.where(inside, at, torch.full_like(at, t.shape[1]))]


def _unpadded(t, st):
    if st["offsets"] is None:
        return t[:, :st["case"]["L"]]
    at = st["offsets"][:-1, None].long() + torch.arange(t.shape[1], device=t.device)
    return t[at < st["offsets"][1:, None]].unsqueeze(0)


def _unit(t, on):
    if not on:
        return t, None
    r = torch.rsqrt(t.square().sum(-1, keepdim=True) + _EPS_L2)
    return t * r, r


def _plain_chunks(st):
    """The chunks' products that need no state: [B, H, chunks, 64, ...]."""
    case = st["case"]
    H, share = case["H"], case["H"] // case["Hk"]
    pad = -(-max(1, st["max_len"]) // _CHUNK) * _CHUNK
    heads = lambda t: t.unflatten(1, (pad // _CHUNK, _CHUNK)).movedim(3, 1)
    q, rq = _unit(heads(_padded(st["q"], st, pad)), case["l2norm"])
    k, rk = _unit(heads(_padded(st["k"], st, pad)), case["l2norm"])
    wide = lambda t: t if t is None or share == 1 else t.repeat_interleave(share, dim=1)
    c = {"q": wide(q) / math.sqrt(case["dk"]), "k": wide(k), "qu": q, "ku": k, "rq": rq, "rk": rk, "pad": pad}
    c["v"] = heads(_padded(st["v"], st, pad))
    beta = heads(_padded(st["beta"].unsqueeze(-1), st, pad))
    G = heads(_padded(st["g"].unsqueeze(-1), st, pad)).cumsum(-2)
    lower = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=G.device).tril()
    D = torch.where(lower, G - G.transpose(-1, -2), torch.full((), -math.inf, device=G.device)).exp()
    kk = c["k"] @ c["k"].transpose(-1, -2).contiguous()
    M = (beta * D * kk).tril(-1)
    T = torch.zeros_like(M)
    T[..., 0, 0] = 1
    for i in range(1, _CHUNK):  # the inverse of I + M, row by row
        T[..., i, :i] = -(M[..., i:i + 1, :i] @ T[..., :i, :i]).squeeze(-2)
        T[..., i, i] = 1
    A = c["q"] @ c["k"].transpose(-1, -2).contiguous() * D
    c.update(beta=beta, eG=G.exp(), eR=(G[..., -1:, :] - G).exp(), eC=G[..., -1:, :].exp(), D=D, kk=kk, M=M, T=T, A=A)
    return c


def _plain_states(st, c, outputs):
    """The pass over the chunks: the state before each, U, and (for the forward) the outputs."""
    case = st["case"]
    S = st["h0"].clone() if st["h0"] is not None else torch.zeros(case["B"], case["H"], case["dk"], case["dv"], device="cuda")
    before, us, os = [], [], []
    for n in range(c["pad"] // _CHUNK):
        k, q, eG = c["k"][:, :, n], c["q"][:, :, n], c["eG"][:, :, n]
        U = c["T"][:, :, n] @ (c["beta"][:, :, n] * (c["v"][:, :, n] - eG * (k @ S)))
        if outputs:
            os.append(eG * (q @ S) + c["A"][:, :, n] @ U)
        else:
            before.append(S)
            us.append(U)
        S = c["eC"][:, :, n] * S + (k * c["eR"][:, :, n]).transpose(-1, -2).contiguous() @ U
    return S, before, us, os


def _plain_fwd(st):
    c = _plain_chunks(st)
    S, _, _, os = _plain_states(st, c, True)
    o = torch.cat(os, dim=2).movedim(1, 2)
    o = _unpadded(o, st).contiguous().to(_TYPES[st["case"]["io"]])
    return {"o": o, "state": S} if st["case"]["state"] else {"o": o}


def _plain_bwd(st):
    case = st["case"]
    c = _plain_chunks(st)
    _, before, us, _ = _plain_states(st, c, False)
    tr = lambda t: t.transpose(-1, -2).contiguous()
    dO = _padded(st["do"], st, c["pad"]).unflatten(1, (-1, _CHUNK)).movedim(3, 1)
    dS = torch.zeros(case["B"], case["H"], case["dk"], case["dv"], device="cuda")
    got = []
    for n in reversed(range(c["pad"] // _CHUNK)):
        q, k, v, beta, eG, eR, eC, D, kk, M, T, A = (c[m][:, :, n] for m in ("q", "k", "v", "beta", "eG", "eR", "eC", "D", "kk", "M", "T", "A"))
        S, U, do = before[n], us[n], dO[:, :, n]
        kdS = (k * eR) @ dS
        dR = tr(T) @ (tr(A) @ do + kdS)
        rest = v - eG * (k @ S)
        dM = -(dR @ tr(U)).tril(-1)
        dA = (do @ tr(U)).tril()
        W, P, E = dM * beta * D, dA * A, dM * M
        dks = -beta * eG * dR
        dos = eG * do
        dq = (dos @ tr(S) + (dA * D) @ k) / math.sqrt(case["dk"])
        dk = dks @ tr(S) + (U * eR) @ tr(dS) + tr(dA * D) @ q + W @ k + tr(W) @ k
        dbeta = (dR * rest).sum(-1) + (dM * D * kk).sum(-1)
        through = (kdS * U).sum(-1)
        dG = P.sum(-1) - P.sum(-2) + E.sum(-1) - E.sum(-2) + (dks * (k @ S)).sum(-1) + (dos * (q @ S)).sum(-1) - through
        dG[..., -1] += through.sum(-1) + (eC * dS * S).sum((-1, -2))
        got.append((dq, dk, beta * dR, dG.flip(-1).cumsum(-1).flip(-1).unsqueeze(-1), dbeta.unsqueeze(-1)))
        dS = eC * dS + tr(q) @ dos + tr(k) @ dks
    dq, dk, dv, dg, db = (torch.stack(t[::-1], dim=2) for t in zip(*got))
    share = lambda t: t.unflatten(1, (case["Hk"], -1)).sum(2)
    dq, dk = share(dq), share(dk)
    if case["l2norm"]:
        dq = c["rq"] * (dq - c["qu"] * (dq * c["qu"]).sum(-1, keepdim=True))
        dk = c["rk"] * (dk - c["ku"] * (dk * c["ku"]).sum(-1, keepdim=True))
    io = _TYPES[case["io"]]
    back = lambda t: _unpadded(t.movedim(1, 3).flatten(1, 2), st).contiguous().to(io)
    out = {"dq": back(dq), "dk": back(dk), "dv": back(dv), "dg": back(dg).squeeze(-1), "dbeta": back(db).squeeze(-1)}
    if st["h0"] is not None:
        out["dh0"] = dS
    return out


def _plain_step(st):
    case = st["case"]
    share = case["H"] // case["Hk"]
    q, k = _unit(st["q"].float(), case["l2norm"])[0], _unit(st["k"].float(), case["l2norm"])[0]
    q, k = (t.repeat_interleave(share, dim=1).unsqueeze(-1) for t in (q / math.sqrt(case["dk"]), k))
    S = st["pool"][st["slots"].long()] * st["g"].float().exp()[..., None, None]
    u = st["beta"].float().unsqueeze(-1) * (st["v"].float() - (k * S).sum(-2))
    S = S + k * u.unsqueeze(-2)
    st["pool"][st["slots"].long()] = S
    return {"o": (q * S).sum(-2).to(_TYPES[case["io"]]), "pool": st["pool"]}


def _plain_gn(st):
    case = st["case"]
    N, L, C, G = case["N"], case["L"], case["C"], case["G"]
    x = st["x"].float().view(N, L, G, C // G)
    mean = x.mean(dim=(1, 3))
    rstd = torch.rsqrt((x - mean.view(N, 1, G, 1)).square().mean(dim=(1, 3)) + _EPS_GN)
    z = ((x - mean.view(N, 1, G, 1)) * rstd.view(N, 1, G, 1)).view(N, L, C)
    if case["affine"]:
        z = z * st["w"] + st["b"]
    if case["act"] == "silu":
        z = z / (1 + (-z).exp())
    return {"y": z.to(st["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_gn_bwd(st):
    case = st["case"]
    N, L, C, G = case["N"], case["L"], case["C"], case["G"]
    mean, rstd = st["mean"].view(N, 1, G, 1), st["rstd"].view(N, 1, G, 1)
    xh = (st["x"].float().view(N, L, G, C // G) - mean) * rstd
    dz = st["dy"].float()
    if case["act"] == "silu":
        z = xh.view(N, L, C)
        if case["affine"]:
            z = z * st["w"] + st["b"]
        s = 1 / (1 + (-z).exp())
        dz = dz * (s * (1 + z * (1 - s)))
    out = {}
    if case["affine"]:
        out["dw"], out["db"] = (dz * xh.view(N, L, C)).sum(dim=1).sum(dim=0), dz.sum(dim=1).sum(dim=0)
        dz = dz * st["w"]
    dz = dz.view(N, L, G, C // G)
    dx = rstd * (dz - dz.mean(dim=(1, 3), keepdim=True) - xh * (dz * xh).mean(dim=(1, 3), keepdim=True))
    out["dx"] = dx.view(N, L, C).to(st["x"].dtype)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"gdr_fwd": _plain_fwd, "gdr_bwd": _plain_bwd, "gdr_step": _plain_step, "gn_fwd": _plain_gn,
                "gn_bwd": _plain_gn_bwd}[op](state)
    import selective_scan_segmented_amd as sfm
    s = state
    if op == "gdr_fwd":
        got = sfm.sfm_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"], offsets=s["offsets"],
                                      max_len=s["max_len"], l2norm=case["l2norm"], return_state=case["state"])
        return {"o": got[0], "state": got[1]} if case["state"] else {"o": got}
    if op == "gdr_bwd":
        return sfm.sfm_gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], h0=s["h0"],
                                       offsets=s["offsets"], max_len=s["max_len"], l2norm=case["l2norm"])
    if op == "gdr_step":
        o = sfm.sfm_gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], slots=s["slots"],
                                     l2norm=case["l2norm"])
        return {"o": o, "pool": s["pool"]}
    if op == "gn_fwd":
        y, mean, rstd = sfm.sfm_group_norm_fwd(s["x"], case["G"], s["w"], s["b"], eps=_EPS_GN, act=case["act"])
        return {"y": y, "mean": mean, "rstd": rstd}
    return sfm.sfm_group_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], s["b"], act=case["act"])


def work(case):
    e = 4 if case["io"] == "f32" else 2
    if case["op"].startswith("gn"):
        n = case["N"] * case["L"] * case["C"]
        stats, affine = 8 * case["N"] * case["G"], 8 * case["C"] * case["affine"]
        if case["op"] == "gn_fwd":  # two operations for the sums, three to apply them, four for the activation
            return {"bytes": 2 * n * e + stats + affine, "flops": n * (9 if case["act"] == "silu" else 5)}
        return {"bytes": 3 * n * e + stats + 2 * affine, "flops": n * (18 if case["act"] == "silu" else 10)}
    Hk, H, dk, dv = (case[n] for n in ("Hk", "H", "dk", "dv"))
    if case["op"] == "gdr_step":
        B = case["B"]
        return {"bytes": B * (e * (2 * Hk * dk + 2 * H * dv + 2 * H) + 8 * H * dk * dv + 4), "flops": 7 * B * H * dk * dv}
    tokens = sum(_lengths(case))
    state = 4 * case["B"] * H * dk * dv
    row = 2 * Hk * dk + H * dv + 2 * H
    if case["op"] == "gdr_fwd":  # S^T k, the rank-one update, the decay and S^T q of each token
        return {"bytes": tokens * e * (row + H * dv) + state * (case["h0"] + case["state"]), "flops": 7 * tokens * H * dk * dv}
    # the states again (5), q and k's gradients from the state and its gradient, du, dr, the decay's gradient
    return {"bytes": tokens * e * (2 * row + H * dv) + state * 2 * case["h0"], "flops": 18 * tokens * H * dk * dv}


# ---------------------------------------------------------------- the definitions, in 64 bits
def _double(t):
    return None if t is None else t.double()


def _norm64(t, on):
    return t / (t.pow(2).sum(-1, keepdim=True) + _EPS_L2).sqrt() if on else t


def _token(t, st, i):
    """Token i of every row (those that have one) of [B, L, ...] or packed [1, total, ...]."""
    if st["offsets"] is None:
        return t[:, i]
    return t[0, (st["offsets"][:-1].long() + i).clamp(max=t.shape[1] - 1)]


def _recurrence(st, S, first, last, keep):
    """Tokens first .. last - 1 of every row by the definition; `keep` takes what each token saw."""
    case = st["case"]
    share = case["H"] // case["Hk"]
    lens = torch.tensor(_lengths(case), device=S.device)
    for i in range(first, last):
        live = (lens > i).view(-1, 1, 1, 1)
        q, k, v, g, beta = (_token(st[n], st, i).double() for n in ("q", "k", "v", "g", "beta"))
        q, k = (_norm64(t, case["l2norm"]).repeat_interleave(share, dim=1) for t in (q, k))
        a = g.exp()[..., None, None]
        r = v - (a * S * k.unsqueeze(-1)).sum(-2)
        u = beta.unsqueeze(-1) * r
        after = torch.where(live, a * S + k.unsqueeze(-1) * u.unsqueeze(-2), S)
        keep(i, live, q, k, a, beta, r, u, S, after)
        S = after
    return S


def _put(out, st, i, value):
    if st["offsets"] is None:
        out[:, i] = value
        return
    lens = st["offsets"][1:] - st["offsets"][:-1]
    rows = (lens > i).nonzero().flatten()
    out[0, st["offsets"][:-1].long()[rows] + i] = value[rows]


def _exact_fwd(st):
    case = st["case"]
    o = torch.zeros(st["v"].shape, dtype=torch.float64, device="cuda")
    S = _double(st["h0"]) if st["h0"] is not None else torch.zeros(case["B"], case["H"], case["dk"], case["dv"], dtype=torch.float64, device="cuda")
    keep = lambda i, live, q, k, a, beta, r, u, S0, S1: _put(o, st, i, (q.unsqueeze(-1) * S1).sum(-2) / math.sqrt(case["dk"]))
    S = _recurrence(st, S, 0, max(_lengths(case)), keep)
    return {"o": o, "state": S} if case["state"] else {"o": o}


def _exact_bwd(st):
    case = st["case"]
    share, scale, most = case["H"] // case["Hk"], 1 / math.sqrt(case["dk"]), max(_lengths(case))
    zero = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
    S = _double(st["h0"]) if st["h0"] is not None else torch.zeros(case["B"], case["H"], case["dk"], case["dv"], dtype=torch.float64, device="cuda")
    starts = []
    for n in range(0, most, 32):
        starts.append((n, S))
        S = _recurrence(st, S, n, min(most, n + 32), lambda *a: None)
    out = {"dq": zero(st["q"]), "dk": zero(st["k"]), "dv": zero(st["v"]), "dg": zero(st["g"]), "dbeta": zero(st["beta"])}
    dS = torch.zeros_like(S)

    def raw(d, name, i):
        d = d.unflatten(1, (case["Hk"], share)).sum(2)
        if case["l2norm"]:
            x = _token(st[name], st, i).double()
            n = (x.pow(2).sum(-1, keepdim=True) + _EPS_L2).sqrt()
            d = d / n - x * (x * d).sum(-1, keepdim=True) / n ** 3
        return d

    for n, S in reversed(starts):
        seen = []
        _recurrence(st, S, n, min(most, n + 32), lambda *a: seen.append(a))
        while seen:
            i, live, q, k, a, beta, r, u, S0, S1 = seen.pop()
            do = _token(st["do"], st, i).double()
            at = dS + scale * q.unsqueeze(-1) * do.unsqueeze(-2)
            du = (at * k.unsqueeze(-1)).sum(-2)
            dr = beta.unsqueeze(-1) * du
            _put(out["dq"], st, i, raw(scale * (S1 * do.unsqueeze(-2)).sum(-1), "q", i))
            _put(out["dk"], st, i, raw((at * u.unsqueeze(-2)).sum(-1) - (a * S0 * dr.unsqueeze(-2)).sum(-1), "k", i))
            _put(out["dv"], st, i, dr)
            _put(out["dbeta"], st, i, (du * r).sum(-1))
            before = at - k.unsqueeze(-1) * dr.unsqueeze(-2)
            _put(out["dg"], st, i, (a * before * S0).sum((-1, -2)))
            dS = torch.where(live, a * before, dS)
    if st["h0"] is not None:
        out["dh0"] = dS
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("gn"):
        N, L, C, G = case["N"], case["L"], case["C"], case["G"]
        x = st["x"].double().reshape(N, L, G, -1)
        affine = (lambda t: t * _double(st["w"]) + _double(st["b"])) if case["affine"] else (lambda t: t)
        if case["op"] == "gn_fwd":
            var, mean = torch.var_mean(x, dim=(1, 3), correction=0, keepdim=True)
            z = affine(((x - mean) / (var + _EPS_GN).sqrt()).reshape(N, L, C))
            y = z * torch.sigmoid(z) if case["act"] == "silu" else z
            return {"y": y, "mean": mean.reshape(N, G), "rstd": (var + _EPS_GN).rsqrt().reshape(N, G)}
        mean, rstd = st["mean"].double().view(N, 1, G, 1), st["rstd"].double().view(N, 1, G, 1)
        xh = ((x - mean) * rstd).reshape(N, L, C)
        z, d = affine(xh), st["dy"].double()
        if case["act"] == "silu":
            s = torch.sigmoid(z)
            d = d * s * (1 + z * (1 - s))
        out = {"dw": (d * xh).sum((0, 1)), "db": d.sum((0, 1))} if case["affine"] else {}
        d = (d * _double(st["w"]) if case["affine"] else d).reshape(N, L, G, -1)
        xh = xh.reshape(N, L, G, -1)
        out["dx"] = (rstd * (d - d.mean((1, 3), keepdim=True) - xh * (d * xh).mean((1, 3), keepdim=True))).reshape(N, L, C)
        return out
    if case["op"] == "gdr_fwd":
        return _exact_fwd(st)
    if case["op"] == "gdr_bwd":
        return _exact_bwd(st)
    share = case["H"] // case["Hk"]
    q, k = (_norm64(st[n].double(), case["l2norm"]).repeat_interleave(share, dim=1) for n in ("q", "k"))
    rows = st["slots"].long()
    S = st["pool"][rows].double() * st["g"].double().exp()[..., None, None]
    u = st["beta"].double().unsqueeze(-1) * (st["v"].double() - (k.unsqueeze(-1) * S).sum(-2))
    S = S + k.unsqueeze(-1) * u.unsqueeze(-2)
    pool = st["pool"].double()
    pool[rows] = S
    return {"o": (q.unsqueeze(-1) * S).sum(-2) / math.sqrt(case["dk"]), "pool": pool}
