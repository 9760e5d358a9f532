"""Measured cases of the gated delta rule and of the cell-output layer norm.

Gated delta rule, per (batch, head), with the state C of d_qk x d_v (fp32):

    C_t = e^{g_t} C_{t-1} + beta_t k_t (v_t - e^{g_t} C_{t-1}^T k_t)^T
    h_t = scale * C_t^T q_t,            scale = 1 / sqrt(d_qk)

``g`` is the log decay (<= 0), ``beta`` the writing strength.  Q and K may have
fewer heads than V (head n of V reads head n // (NH / NHK) of Q and K).

Cell-output layer norm: the output X [B, NH, T, D] of the cell is normalised
over D per (token, head), scaled and shifted per (head, column) and laid out
token-major, Y [B, T, NH * D].  With NH = 1 it is the layer norm of rows.

Kinds of cases: "fw" the chunkwise forward with the final state, "train" the
forward and the gradients of every input through autograd, "step" one token in
place on the state, "norm_fw" and "norm_bw" the two halves of the layer norm,
"norm_train" both through autograd.
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 64  # chunk length of the plain form

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cell(name, kind, B, NHK, NH, T, DK, DV, dtype="bf16", init=False):
    return {"name": name, "kind": kind, "B": B, "NHK": NHK, "NH": NH, "T": T, "DK": DK, "DV": DV,
            "dtype": dtype, "init": init}


def _norm(name, kind, B, NH, T, D, dtype="bf16", bias=True):
    return {"name": name, "kind": kind, "B": B, "NH": NH, "T": T, "D": D, "dtype": dtype,
            "bias": bias}


def listed():
    return [
        # four short prompts of a small model: the call is all latency
        _cell("fw_short", "fw", 4, 4, 4, 77, 64, 64),
        # the mid workload's shape: a batch of two, 4096 tokens
        _cell("fw_mid", "fw", 2, 8, 8, 4096, 128, 128),
        # one long prompt of odd length that continues a state; two value heads per key head
        _cell("fw_shared_long", "fw", 1, 8, 16, 8191, 128, 128, init=True),
        # a point of the chunk / length sweep: 65536 tokens, 256 heads; the largest forward
        _cell("fw_sweep", "fw", 16, 16, 16, 4096, 128, 128),
        # fp32 inputs, value rows that are no multiple of a tile
        _cell("fw_f32", "fw", 1, 4, 4, 1000, 64, 96, dtype="f32", init=True),
        # a training micro-batch of odd length
        _cell("train_mid", "train", 2, 8, 8, 2047, 128, 128),
        # a training batch with shared key heads and a carried-in state
        _cell("train_shared", "train", 2, 8, 16, 4096, 128, 128, init=True),
        # decoding: one sequence, and a batch that fills the GPU
        _cell("step_one", "step", 1, 16, 16, 1, 128, 128, init=True),
        _cell("step_batch", "step", 96, 8, 16, 1, 128, 128, init=True),
        # the cell output of the 7B-shaped batch (8 heads of 512 columns)
        _norm("norm_fw_7b", "norm_fw", 8, 8, 8192, 512),
        # its gradients
        _norm("norm_bw_7b", "norm_bw", 8, 8, 8192, 512),
        # the norm before a block: rows of the model's width, forward and backward, odd row count
        _norm("norm_train_rows", "norm_train", 3, 1, 333, 2048),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["fw", "fw", "train", "train", "step", "norm_fw", "norm_bw", "norm_train"])
    if kind.startswith("norm"):
        D = rng.choice([64, 96, 128, 256, 512, 768, 1024, 2048, 4096])
        NH = rng.choice([1, 2, 4, 8, 12, 16]) if D <= 512 else 1
        B = rng.choice([1, 2, 3, 4, 8])
        T = _log_int(rng, 1, min(16384, max(1, (1 << 27) // (B * NH * D))))
        case = _norm("", kind, B, NH, T, D, dtype=rng.choice(["bf16", "bf16", "f32"]),
                     bias=rng.random() < 0.7)
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        DK = rng.choice([64, 96, 128])
        DV = rng.choice([64, 96, 128, 256])
        NHK = rng.choice([1, 2, 4, 8, 16])
        NH = NHK * rng.choice([1, 1, 2, 4])
        if kind == "step":
            B, T = _log_int(rng, 1, max(1, 1536 // NH)), 1
        else:
            B = _log_int(rng, 1, 8)
            # the largest: 2^20 (train: 2^17, fp32 inputs: an eighth) head-tokens
            most = 1 << (20 if kind == "fw" else 17)
            if dtype == "f32":
                most >>= 3
            T = _log_int(rng, 1, max(1, min(16384, most // (B * NH) * 128 // max(DV, 128))))
        case = _cell("", kind, B, NHK, NH, T, DK, DV, dtype=dtype,
                     init=kind == "step" or rng.random() < 0.5)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dt = _DT[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["kind"].startswith("norm"):
        B, NH, T, D = case["B"], case["NH"], case["T"], case["D"]
        s = {"X": (randn(B, NH, T, D) + 0.3 * randn(B, NH, T, 1)).to(dt),
             "weight": 1.0 + 0.1 * randn(NH, D),
             "bias": 0.1 * randn(NH, D) if case["bias"] else None}
        if case["kind"] != "norm_fw":
            s["dY"] = randn(B, T, NH * D).to(dt)
        if case["kind"] == "norm_bw":  # what the forward pass kept
            X = s["X"].double()
            mean = X.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = ((X - mean[..., None]).square().mean(-1) + EPS).rsqrt().float()
        return {"case": case, **s}

    B, NHK, NH, T, DK, DV = (case[n] for n in ("B", "NHK", "NH", "T", "DK", "DV"))

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).sqrt()

    # unit queries and keys; decay rates spread over the heads as the usual parametrisation
    # -A softplus(x + bias) gives them: from almost none to a few tokens
    rate = torch.exp(torch.linspace(math.log(2e-3), math.log(0.8), NH, device="cuda"))
    s = {"Q": unit(randn(B, NHK, T, DK)).to(dt), "K": unit(randn(B, NHK, T, DK)).to(dt),
         "V": randn(B, NH, T, DV).to(dt),
         "g": -rate[None, :, None] * torch.exp(0.5 * randn(B, NH, T)),
         "beta": torch.sigmoid(randn(B, NH, T)),
         "C0": 0.3 * randn(B, NH, DK, DV) if case["init"] else None}
    if case["kind"] == "train":
        s["dH"] = randn(B, NH, T, DV).to(dt)
        for n in ("Q", "K", "V", "g", "beta", "C0"):
            if s[n] is not None:
                s[n].requires_grad_()
    if case["kind"] == "step":
        for n in ("Q", "K", "V", "g", "beta"):
            s[n] = s[n].squeeze(2).contiguous()
    return {"case": case, **s}


# ------------------------------------------------------- the plain forms
def _unit_lower_inverse(A):
    """(I + A)^{-1} of strictly lower triangular A, by doubling the block size:
    the inverse's lower left block is -T22 A21 T11."""
    n = A.shape[-1]
    idx = torch.arange(n, device=A.device)
    X = torch.eye(n, device=A.device, dtype=A.dtype).expand(A.shape)
    s = 1
    while s < n:
        blk = idx // s
        pair = (blk[:, None] % 2 == 1) & (blk[None, :] == blk[:, None] - 1)
        X = X - X @ torch.where(pair, A, 0.0) @ X
        s *= 2
    return X


def _plain_fw(Q, K, V, g, beta, C0):
    """Chunkwise, in 32 bits: per chunk y = (I + A)^{-1} (V - e^gc K C) with
    A_rs = e^{gc_r - gc_s} beta_s k_r.k_s (s < r), then h and the next state."""
    B, NH, T, DV = V.shape
    DK, L = Q.shape[-1], CHUNK
    scale = DK ** -0.5
    per = NH // Q.shape[1]
    NC = -(-T // L)

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0, 0, NC * L - T))
        return x.reshape(B, NH, NC, L, x.shape[-1])

    Q, K = (chunks(x.float().repeat_interleave(per, dim=1)) for x in (Q, K))
    V, beta = chunks(V.float()), chunks(beta.float()[..., None])
    gc = chunks(g.double()[..., None])[..., 0].cumsum(-1)  # 64 bits: differences of long sums
    lower = torch.ones(L, L, device=V.device).tril().bool()
    diff = torch.where(lower, gc[..., :, None] - gc[..., None, :], 0.0)
    decay = torch.where(lower, torch.exp(diff).float(), 0.0)
    from_start = torch.exp(gc).float()[..., None]
    to_end = torch.exp(gc[..., -1:] - gc).float()[..., None]
    W = decay * beta.transpose(-1, -2)
    inv = _unit_lower_inverse((W * (K @ K.transpose(-1, -2))).tril(-1))
    P = W * (Q @ K.transpose(-1, -2))
    C = torch.zeros(B, NH, DK, DV, device=V.device) if C0 is None else C0.float()
    out = []
    for c in range(NC):
        Kc, lam = K[:, :, c], from_start[:, :, c]
        y = inv[:, :, c] @ (V[:, :, c] - lam * (Kc @ C))
        out.append(scale * (lam * (Q[:, :, c] @ C) + P[:, :, c] @ y))
        C = lam[:, :, -1:] * C + Kc.transpose(-1, -2) @ (to_end[:, :, c] * beta[:, :, c] * y)
    return torch.cat(out, 2)[:, :, :T], C


def _plain_step(s):
    q, k, v, C = (s[n].float() for n in ("Q", "K", "V", "C0"))
    per = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(per, dim=1), k.repeat_interleave(per, dim=1)
    C = torch.exp(s["g"])[..., None, None] * C
    u = s["beta"][..., None] * (v - (C * k[..., None]).sum(-2))
    C = C + k[..., None] * u[..., None, :]
    s["C0"].copy_(C)
    h = q.shape[-1] ** -0.5 * (C * q[..., None]).sum(-2)
    return {"h": h.to(s["V"].dtype), "C": s["C0"]}


def _token_major(x):
    B, NH, T, D = x.shape
    return x.transpose(1, 2).reshape(B, T, NH * D)


def _plain_norm_fw(X, weight, bias):
    x = X.float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = 1.0 / (d.square().mean(-1, keepdim=True) + EPS).sqrt()
    y = d * rstd * weight[None, :, None, :]
    if bias is not None:
        y = y + bias[None, :, None, :]
    return _token_major(y).to(X.dtype), mean[..., 0], rstd[..., 0]


def _plain_norm_bw(s):
    X, w = s["X"].float(), s["weight"]
    B, NH, T, D = X.shape
    dy = s["dY"].float().reshape(B, T, NH, D).transpose(1, 2)
    xh = (X - s["mean"][..., None]) * s["rstd"][..., None]
    a = dy * w[None, :, None, :]
    dx = s["rstd"][..., None] * (a - a.mean(-1, keepdim=True)
                                 - xh * (a * xh).mean(-1, keepdim=True))
    out = {"dX": dx.to(s["X"].dtype), "dweight": (dy * xh).sum((0, 2))}
    if s["bias"] is not None:
        out["dbias"] = dy.sum((0, 2))
    return out


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "fw":
        H, C = _plain_fw(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["C0"])
        return {"H": H.to(s["V"].dtype), "C_T": C}
    if kind == "train":
        names = [n for n in ("Q", "K", "V", "g", "beta", "C0") if s[n] is not None]
        H, _ = _plain_fw(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["C0"])
        H = H.to(s["V"].dtype)
        grads = torch.autograd.grad(H, [s[n] for n in names], s["dH"])
        return {"H": H.detach(), **{"d" + n: x for n, x in zip(names, grads)}}
    if kind == "step":
        return _plain_step(s)
    if kind == "norm_fw":
        Y, mean, rstd = _plain_norm_fw(s["X"], s["weight"], s["bias"])
        return {"Y": Y, "mean": mean, "rstd": rstd}
    if kind == "norm_bw":
        return _plain_norm_bw(s)
    Y, mean, rstd = _plain_norm_fw(s["X"], s["weight"], s["bias"])
    return {"Y": Y, **_plain_norm_bw({**s, "mean": mean, "rstd": rstd})}


# ------------------------------------------------- the framework's calls
def _own(s):
    from mlstm_chunkwise_b200 import api

    kind = s["case"]["kind"]
    if kind == "fw":
        H, C_T = api.gated_delta_fw(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["C0"])
        return {"H": H, "C_T": C_T}
    if kind == "train":
        names = [n for n in ("Q", "K", "V", "g", "beta", "C0") if s[n] is not None]
        H, _ = api.gated_delta_chunkwise(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["C0"])
        grads = torch.autograd.grad(H, [s[n] for n in names], s["dH"])
        return {"H": H.detach(), **{"d" + n: x for n, x in zip(names, grads)}}
    if kind == "step":
        h = api.gated_delta_step(s["Q"], s["K"], s["V"], s["g"], s["beta"], s["C0"])
        return {"h": h, "C": s["C0"]}
    if kind == "norm_fw":
        Y, mean, rstd = api.head_norm_fw(s["X"], s["weight"], s["bias"], eps=EPS)
        return {"Y": Y, "mean": mean, "rstd": rstd}
    if kind == "norm_bw":
        return api.head_norm_bw(s["X"], s["dY"], s["weight"], s["mean"], s["rstd"],
                                bias=s["bias"] is not None)
    X, w, b = (None if s[n] is None else s[n].detach().requires_grad_()
               for n in ("X", "weight", "bias"))
    Y = api.head_norm(X, w, b, eps=EPS)
    leaves = [X, w] if b is None else [X, w, b]
    grads = torch.autograd.grad(Y, leaves, s["dY"])
    return {"Y": Y.detach(), **dict(zip(("dX", "dweight", "dbias"), grads))}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["kind"].startswith("norm"):
        n = case["B"] * case["NH"] * case["T"] * case["D"]
        rows = n // case["D"]
        params = 4 * case["NH"] * case["D"] * (2 if case["bias"] else 1)
        by = {"norm_fw": 2 * esz * n + 8 * rows + params,
              "norm_bw": 3 * esz * n + 8 * rows + 4 * case["NH"] * case["D"] + params,
              "norm_train": 4 * esz * n + 2 * params}[case["kind"]]
        return {"bytes": by, "flops": {"norm_fw": 7, "norm_bw": 13, "norm_train": 20}[case["kind"]] * n}
    B, NHK, NH, T, DK, DV = (case[n] for n in ("B", "NHK", "NH", "T", "DK", "DV"))
    qk, v = esz * B * NHK * T * DK, esz * B * NH * T * DV
    gates, state = 8 * B * NH * T, 4 * B * NH * DK * DV
    # per token and head: C^T k, the rank-one update and C^T q; the gradients: the two rank-one
    # updates of dC, its products with k and y, the products of C with dh and dy, and <C, dC>
    if case["kind"] == "train":
        by = 4 * qk + 4 * v + 2 * gates + (2 * state if case["init"] else 0)
        return {"bytes": by, "flops": 20 * B * NH * T * DK * DV}
    by = 2 * qk + 2 * v + gates + state + (state if case["init"] else 0)
    return {"bytes": by, "flops": 6 * B * NH * T * DK * DV}


# ----------------------------------------- the definition, in 64 bits
def _exact_norm(s, kind):
    X, w = s["X"].double(), s["weight"].double()
    B, NH, T, D = X.shape
    mean = X.mean(-1)
    rstd = (((X * X).mean(-1) - mean * mean) + EPS) ** -0.5
    if kind == "norm_bw":
        mean, rstd = s["mean"].double(), s["rstd"].double()
    xh = torch.einsum("bhtd,bht->bhtd", X - mean[..., None], rstd)
    out = {}
    if kind != "norm_bw":
        Y = torch.einsum("bhtd,hd->bthd", xh, w)
        if s["bias"] is not None:
            Y = Y + s["bias"].double()
        out["Y"] = Y.reshape(B, T, NH * D)
    if kind == "norm_fw":
        out.update(mean=mean, rstd=rstd)
        return out
    dy = s["dY"].double().view(B, T, NH, D)
    a = torch.einsum("bthd,hd->bhtd", dy, w)
    dot = torch.einsum("bhtd,bhtd->bht", a, xh) / D
    out["dX"] = (a - a.mean(-1, keepdim=True) - xh * dot[..., None]) * rstd[..., None]
    out["dweight"] = torch.einsum("bthd,bhtd->hd", dy, xh)
    if s["bias"] is not None:
        out["dbias"] = dy.sum((0, 1))
    return out


def _exact_cell(s, kind):
    """Token by token.  The gradients run the recurrence backwards over stored
    stretches of states."""
    step = kind == "step"
    Q, K, V, g, beta = (s[n].detach().double() for n in ("Q", "K", "V", "g", "beta"))
    if step:
        Q, K, V, g, beta = (x.unsqueeze(2) for x in (Q, K, V, g, beta))
    B, NH, T, DV = V.shape
    NHK, DK = Q.shape[1], Q.shape[3]
    scale = 1.0 / math.sqrt(DK)
    head = torch.arange(NH, device=V.device) // (NH // NHK)
    Q, K = Q[:, head], K[:, head]
    a = torch.exp(g)
    C = (torch.zeros(B, NH, DK, DV, device=V.device, dtype=torch.float64) if s["C0"] is None
         else s["C0"].detach().double())
    H = torch.empty_like(V)
    keep, L = [], 32

    def advance(C, t):
        C = a[:, :, t, None, None] * C
        y = V[:, :, t] - (K[:, :, t, None, :] @ C).squeeze(-2)
        return C + K[:, :, t, :, None] * (beta[:, :, t, None] * y)[:, :, None, :], y

    for t in range(T):
        if kind == "train" and t % L == 0:
            keep.append(C)
        C, _ = advance(C, t)
        H[:, :, t] = scale * (Q[:, :, t, None, :] @ C).squeeze(-2)
    if step:
        return {"h": H[:, :, 0], "C": C}
    if kind == "fw":
        return {"H": H, "C_T": C}
    dH = s["dH"].double()
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    dC = torch.zeros_like(C)
    for c in reversed(range(len(keep))):
        Cs, ys = [keep[c]], []
        for t in range(c * L, min(T, c * L + L)):
            Cn, y = advance(Cs[-1], t)
            Cs.append(Cn)
            ys.append(y)
        for t in reversed(range(c * L, min(T, c * L + L))):
            C1, y, d, b, k = Cs[t - c * L + 1], ys[t - c * L], dH[:, :, t], beta[:, :, t], K[:, :, t]
            C0 = a[:, :, t, None, None] * Cs[t - c * L]  # the decayed state
            dQ[:, :, t] = scale * (C1 @ d[..., None]).squeeze(-1)
            dC = dC + scale * Q[:, :, t, :, None] * d[:, :, None, :]
            e = (k[:, :, None, :] @ dC).squeeze(-2)
            dbeta[:, :, t] = (e * y).sum(-1)
            dV[:, :, t] = b[..., None] * e
            dK[:, :, t] = b[..., None] * ((dC @ y[..., None]) - (C0 @ e[..., None])).squeeze(-1)
            dC = dC - k[..., None] * (b[..., None] * e)[:, :, None, :]
            dg[:, :, t] = (C0 * dC).sum((-1, -2))
            dC = a[:, :, t, None, None] * dC
    out = {"H": H, "dV": dV, "dg": dg, "dbeta": dbeta}
    out["dQ"], out["dK"] = (x.view(B, NHK, NH // NHK, T, DK).sum(2) for x in (dQ, dK))
    if s["C0"] is not None:
        out["dC0"] = dC
    return out


def exact(case, seed):
    kind = case["kind"]
    if not kind.startswith("norm") and case["T"] > 12000:
        return None  # token by token this takes too long
    s = prepare(case, seed)
    return _exact_norm(s, kind) if kind.startswith("norm") else _exact_cell(s, kind)
