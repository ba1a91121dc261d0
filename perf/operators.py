"""Cases of the operators around the row-typed FFN in a decoder: LayerNorm
(forward with the residual add, and backward), the attention of one new token
over a paged key-value cache (with the append that fills it) and a
mixture-of-experts layer of row-typed SwiGLU experts for a few tokens.

`run` computes a case in plain torch operations (own = False) or through the
library's entry points (own = True); `exact` computes the same from the
definitions in float64.
"""
import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token of the pilot decoder: the residual add and norm before the FFN
        {"name": "norm_token", "op": "norm_fwd", "M": 1, "d": 768, "x": "f32", "delta": "bf16", "y": "bf16"},
        # the pilot batch, 8 sequences of 1536 positions
        {"name": "norm_pilot", "op": "norm_fwd", "M": 12288, "d": 768, "x": "f32", "delta": "f32", "y": "bf16"},
        # a prefill of 2048 tokens at width 4096 with bf16 activations, no residual operand
        {"name": "norm_4096", "op": "norm_fwd", "M": 2048, "d": 4096, "x": "bf16", "delta": "none", "y": "bf16"},
        # the backward pass of the pilot batch's norm, with the residual path's gradient
        {"name": "norm_bwd_pilot", "op": "norm_bwd", "M": 12288, "d": 768, "x": "f32", "dy": "bf16", "ds": True},
        # an odd width and row count in bf16 (rows that start at any 2-byte address)
        {"name": "norm_bwd_odd", "op": "norm_bwd", "M": 1003, "d": 2047, "x": "bf16", "dy": "bf16", "ds": False},
        # one sequence of the pilot decoder (32 heads of 24) early in a generation
        {"name": "attn_pilot_one", "op": "attn", "B": 1, "H": 32, "Hkv": 32, "D": 24, "page": 64, "lo": 200, "hi": 200,
         "q": "f32", "o": "bf16"},
        # a batch of ragged pilot sequences, one of them just started
        {"name": "attn_pilot_batch", "op": "attn", "B": 8, "H": 32, "Hkv": 32, "D": 24, "page": 64, "lo": 1,
         "hi": 1536, "q": "f32", "o": "f32"},
        # serving: a ragged batch with grouped heads of 128, small pages
        {"name": "attn_grouped", "op": "attn", "B": 32, "H": 32, "Hkv": 8, "D": 128, "page": 16, "lo": 1000,
         "hi": 8192, "q": "bf16", "o": "bf16"},
        # one long context
        {"name": "attn_long", "op": "attn", "B": 1, "H": 32, "Hkv": 8, "D": 128, "page": 64, "lo": 131001,
         "hi": 131001, "q": "bf16", "o": "bf16"},
        # experts of the 2048 -> 768 -> 2048 expert FFN at q = 16, 8 of 128: one token
        {"name": "moe_one", "op": "moe", "n": 1, "law": "Qq", "q": 16, "D": 2048, "F": 768, "E": 128, "k": 8,
         "norm": True, "y": "bf16", "pos": 37},
        # the same experts, a batch of new tokens
        {"name": "moe_sixteen", "op": "moe", "n": 16, "law": "Qq", "q": 16, "D": 2048, "F": 768, "E": 128, "k": 8,
         "norm": True, "y": "bf16", "pos": 1000},
        # pilot-wide experts under the tensor square, 2 of 8, plain softmax weights
        {"name": "moe_pilot", "op": "moe", "n": 5, "law": "Q2xQ2", "q": 4, "D": 768, "F": 1536, "E": 8, "k": 2,
         "norm": False, "y": "f32", "pos": 6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "attn", "moe"])
    if op == "norm_fwd":
        d = _log(rng, 48, 8192)
        return {"op": op, "M": min(_log(rng, 1, 16384), 9_000_000 // d), "d": d, "x": rng.choice(["f32", "bf16"]),
                "delta": rng.choice(["none", "f32", "bf16"]), "y": rng.choice(["f32", "bf16"])}
    if op == "norm_bwd":
        d = _log(rng, 48, 8192)
        return {"op": op, "M": min(_log(rng, 1, 16384), 9_000_000 // d), "d": d, "x": rng.choice(["f32", "bf16"]),
                "dy": rng.choice(["f32", "bf16"]), "ds": rng.random() < 0.5}
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8, 12, 32])
        G = rng.choice([1, 1, 2, 3, 4, 8]) if Hkv > 1 else rng.choice([1, 4, 8, 20])
        D = 8 * rng.randint(2, 20)
        B = _log(rng, 1, 48)
        hi = min(_log(rng, 1, 65536), max(1, 140_000_000 // (B * Hkv * D)))
        lo = rng.choice([hi, max(1, hi // 8), 1])
        return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128]), "lo": lo,
                "hi": hi, "q": rng.choice(["f32", "bf16"]), "o": rng.choice(["f32", "bf16"])}
    law = rng.choice(["Qq", "Qq", "Q2xQ2"])
    q = 4 if law == "Q2xQ2" else rng.choice([1, 2, 8, 16, 32])
    D, F = 16 * q * max(1, rng.randint(160, 2304) // (16 * q)), 16 * q * max(1, rng.randint(96, 1600) // (16 * q))
    k = rng.randint(1, 8)
    E = _log(rng, k, 128)
    while E * D * F > 200_000_000:
        E = max(k, E // 2)
        F = max(16 * q, F - 16 * q)
    n = _log(rng, 1, 24)
    while n * k * D * F * (1.0 if q < 8 else 2.0 / q) > 40_000_000 and n > 1:
        n -= 1
    return {"op": op, "n": n, "law": law, "q": q, "D": D, "F": F, "E": E, "k": k, "norm": rng.random() < 0.5,
            "y": rng.choice(["bf16", "f32"]), "pos": rng.randint(0, 5000)}


# ------------------------------------------------------------------ inputs ---

def _randn(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _lengths(c):
    """Lengths from lo to hi, evenly spread over the sequences, long and short ones mixed."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    at = (np.arange(B, dtype=np.int64) * 7 + B - 1) % B if B % 7 else B - 1 - np.arange(B, dtype=np.int64)
    return lo + (hi - lo) * at // (B - 1) if B > 1 else np.array([hi], dtype=np.int64)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(c)
    if c["op"] in ("norm_fwd", "norm_bwd"):
        M, d = c["M"], c["d"]
        xt = DTYPES[c["x"]]
        # a residual stream: every feature with its own offset and scale
        s["X"] = (torch.randn(M, d, generator=g, device=DEV) * (0.5 + torch.rand(d, generator=g, device=DEV))
                  + 0.5 * torch.randn(d, generator=g, device=DEV)).to(xt)
        s["gamma"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["beta"] = 0.1 * torch.randn(d, generator=g, device=DEV)
        if c["op"] == "norm_fwd":
            s["D"] = None if c["delta"] == "none" else _randn(g, (M, d), 0.3, DTYPES[c["delta"]])
            s["S"] = None if c["delta"] == "none" else torch.empty(M, d, dtype=xt, device=DEV)
            s["Y"] = torch.empty(M, d, dtype=DTYPES[c["y"]], device=DEV)
            s["mean"], s["rstd"] = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        else:
            x = s["X"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
            s["dY"] = _randn(g, (M, d), 0.02, DTYPES[c["dy"]])
            s["dS"] = _randn(g, (M, d), 0.02, xt) if c["ds"] else None
            s["dX"] = torch.empty(M, d, dtype=xt, device=DEV)
            s["dgamma"], s["dbeta"] = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    elif c["op"] == "attn":
        B, H, Hkv, D, page = c["B"], c["H"], c["Hkv"], c["D"], c["page"]
        lens = _lengths(c)
        need = -(-lens // page)
        total, most = int(need.sum()), int(need.max())
        n_pages = total + 3
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).to(DEV)
        j = torch.arange(most, device=DEV)
        have = j[None] < torch.from_numpy(need).to(DEV)[:, None]
        at = (first[:, None] + j[None]).clamp_(max=n_pages - 1)
        s["table"] = torch.where(have, order[at], torch.full_like(order[:1], -1)).contiguous()
        # keys [page id, head, position, feature], values [page id, head, feature, position]; slots behind
        # a sequence's end hold what an earlier sequence left there
        s["Kp"] = _randn(g, (n_pages, Hkv, page, D), 1.0, torch.bfloat16)
        s["Vp"] = _randn(g, (n_pages, Hkv, D, page), 1.0, torch.bfloat16)
        s["qkv"] = _randn(g, (B, (H + 2 * Hkv) * D), 1.0, DTYPES[c["q"]])
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        s["last"] = s["lens"] - 1
        s["most"] = most
        s["O"] = torch.empty(B, H, D, dtype=DTYPES[c["o"]], device=DEV)
    else:
        n, q, D, F, E = c["n"], c["q"], c["D"], c["F"], c["E"]
        s["X"] = _randn(g, (n, D), 1.0, torch.bfloat16)
        s["R"] = _randn(g, (E, D), D ** -0.5, torch.bfloat16)
        # block-packed weights of all experts, one after the other
        s["Wg"] = _randn(g, (E, D * F), D ** -0.5, torch.bfloat16)
        s["Wu"] = _randn(g, (E, D * F), D ** -0.5, torch.bfloat16)
        s["Wd"] = _randn(g, (E, F * D), F ** -0.5, torch.bfloat16)
        s["Y"] = torch.empty(n, D, dtype=DTYPES[c["y"]], device=DEV)
        s["experts"] = torch.empty(n, c["k"], dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(n, c["k"], device=DEV)
    if own and c["op"] != "norm_fwd":
        _workspace(s)
    return s


# ------------------------------------------------------- the library's calls ---

@functools.lru_cache(maxsize=None)
def _moe_plans(law, q, D, F, y):
    import associative_algebra_block_amd as aa
    return (aa.aa_plan_create(law, q, D, F, "pos_mod", 0, "bf16", "bf16"),
            aa.aa_plan_create(law, q, F, D, "pos_mod", 0, "bf16", y))


def _workspace(s):
    """The state's own workspace: calls that share one must not overlap in time,
    and another state may be run on another stream."""
    if "workspace" not in s:
        import associative_algebra_block_amd as aa
        n = 0
        if s["op"] == "norm_bwd":
            n = aa.aa_layernorm_bwd_workspace(s["M"], s["d"])
        elif s["op"] == "attn":
            n = aa.aa_attn_decode_workspace(s["B"], s["H"], s["Hkv"], s["D"], s["page"], s["most"])
        elif s["op"] == "moe":
            up, down = _moe_plans(s["law"], s["q"], s["D"], s["F"], s["y"])
            n = aa.aa_moe_ffn_workspace(up, down, s["E"], s["k"], s["n"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return s["workspace"]


def _run_own(s):
    import associative_algebra_block_amd as aa
    if s["op"] == "norm_fwd":
        aa.aa_layernorm_fwd(s["X"], s["gamma"], s["beta"], s["Y"], s["D"], s["S"], s["mean"], s["rstd"], EPS)
        return [s["Y"], s["S"], s["mean"], s["rstd"]]
    if s["op"] == "norm_bwd":
        aa.aa_layernorm_bwd(s["X"], s["dY"], s["gamma"], s["mean"], s["rstd"], s["dX"], s["dgamma"], s["dbeta"],
                            s["dS"], _workspace(s))
        return [s["dX"], s["dgamma"], s["dbeta"]]
    if s["op"] == "attn":
        B, H, Hkv, D = s["B"], s["H"], s["Hkv"], s["D"]
        Q = s["qkv"][:, : H * D]
        K = s["qkv"][:, H * D : (H + Hkv) * D]
        V = s["qkv"][:, (H + Hkv) * D :]
        aa.aa_kv_append(K, V, s["Kp"], s["Vp"], s["table"], s["last"])
        aa.aa_attn_decode(Q, s["Kp"], s["Vp"], s["table"], s["lens"], s["O"], D ** -0.5, _workspace(s))
        return [s["O"], s["Kp"], s["Vp"]]
    up, down = _moe_plans(s["law"], s["q"], s["D"], s["F"], s["y"])
    aa.aa_moe_ffn_fwd(up, down, s["X"], s["R"], s["Wg"], s["Wu"], s["Wd"], s["Y"], s["k"], s["norm"], s["experts"],
                      s["weights"], _workspace(s), pos_offset=s["pos"])
    return [s["Y"], s["experts"], s["weights"]]


# -------------------------------------------------------------- plain forms ---

def _norm_fwd_plain(s):
    x = s["X"].float()
    S = None
    if s["D"] is not None:
        S = (x + s["D"].float()).to(s["X"].dtype)
        x = S.float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * rstd * s["gamma"] + s["beta"]
    return [y.to(DTYPES[s["y"]]), S, mean[:, 0], rstd[:, 0]]


def _norm_bwd_plain(s):
    x, dy = s["X"].float(), s["dY"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["dS"] is not None:
        dx = dx + s["dS"].float()
    return [dx.to(s["X"].dtype), (dy * xh).sum(0), dy.sum(0)]


def _attn_plain(s):
    B, H, Hkv, D, page = s["B"], s["H"], s["Hkv"], s["D"], s["page"]
    q, k, v = s["qkv"].split([H * D, Hkv * D, Hkv * D], 1)
    table, lens, pos = s["table"].long(), s["lens"].long(), s["last"].long()
    # append: the new token's keys and values go to the last position's slot
    at, slot = table.gather(1, (pos // page)[:, None])[:, 0], pos % page
    s["Kp"][at, :, slot] = k.reshape(B, Hkv, D).to(torch.bfloat16)
    s["Vp"][at, :, :, slot] = v.reshape(B, Hkv, D).to(torch.bfloat16)
    # gather every sequence's pages, mask what lies behind its end
    pages = table.clamp(min=0)
    T = s["most"] * page
    keep = torch.arange(T, device=DEV)[None, None] < lens[:, None, None]                     # [B, 1, T]
    Kf = s["Kp"][pages].permute(0, 2, 1, 3, 4).reshape(B * Hkv, T, D).float()
    p = torch.bmm(Kf, q.reshape(B * Hkv, H // Hkv, D).float().transpose(1, 2).contiguous())  # [B Hkv, T, G]
    del Kf
    p = p.transpose(1, 2).reshape(B, H, T) * (1.0 / math.sqrt(D))
    p = p.masked_fill(~keep, float("-inf"))
    p = torch.exp(p - p.amax(2, keepdim=True))
    p = p / p.sum(2, keepdim=True)
    Vf = s["Vp"][pages].permute(0, 2, 3, 1, 4).reshape(B * Hkv, D, T).float()
    o = torch.bmm(Vf, p.view(B * Hkv, H // Hkv, T).transpose(1, 2).contiguous())             # [B Hkv, D, G]
    return [o.transpose(1, 2).reshape(B, H, D).to(DTYPES[s["o"]]), s["Kp"], s["Vp"]]


def _groups(law, q):
    """Input groups of (row type, output group): indices [q, q, S] and which of them count."""
    g = torch.arange(q, device=DEV)
    i, k, j = g[:, None, None], g[None, :, None], g[None, None, :]
    if law == "Qq":
        T = (j == i) | (j == k)
        S = min(2, q)
    else:
        T = ((j // 2 == i // 2) | (j // 2 == k // 2)) & ((j % 2 == i % 2) | (j % 2 == k % 2))
        S = 4
    idx = torch.argsort(T.to(torch.int32), dim=2, descending=True, stable=True)[:, :, :S]
    return idx, T.gather(2, idx)


def _unpack_blocks(w, bi, bo):
    """[..., bi * bo] packed blocks -> [..., bi, bo] float32."""
    lead = w.shape[:-1]
    w = w.reshape(*lead, bo // 16, bi * 16)
    full = bi // 32 * 512
    nl = len(lead)
    a = w[..., :full].reshape(*lead, bo // 16, bi // 32, 4, 16, 8)
    a = a.permute(*range(nl), nl + 1, nl + 2, nl + 4, nl, nl + 3).reshape(*lead, bi // 32 * 32, bo)
    if bi % 32:
        t = w[..., full:].reshape(*lead, bo // 16, 2, 16, 8)
        t = t.permute(*range(nl), nl + 1, nl + 3, nl, nl + 2).reshape(*lead, 16, bo)
        a = torch.cat([a, t], nl)
    return a.float()


def _project_plain(x, W, experts, types, idx, cnt, q, di, do):
    """Rows x [R, di] through experts' packed weights, row-typed."""
    bi, bo = di // q, do // q
    sel, use = idx[types], cnt[types]                                    # [R, q, S]
    R, S = x.shape[0], sel.shape[2]
    k = torch.arange(q, device=DEV)[None, :, None]
    blocks = W.view(-1, q, q, bi * bo)[experts[:, None, None], sel, k]   # [R, q, S, bi * bo]
    xs = x.view(R, q, bi)[torch.arange(R, device=DEV)[:, None, None], sel] * use[..., None]
    y = torch.bmm(xs.reshape(R * q, 1, S * bi), _unpack_blocks(blocks, bi, bo).reshape(R * q, S * bi, bo))
    return y.view(R, do)


def _moe_plain(s):
    n, q, D, F, k = s["n"], s["q"], s["D"], s["F"], s["k"]
    logits = torch.matmul(s["X"].double(), s["R"].double().t().contiguous())   # 64 bits: the choice is a comparison
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    experts = order.indices[:, :k]
    top = order.values
    e = torch.exp(top - top[:, :1]).float()
    weights = e[:, :k] / (e[:, :k] if s["norm"] else e).sum(1, keepdim=True)
    idx, cnt = _groups(s["law"], q)
    pair = experts.reshape(-1)
    types = ((torch.arange(n, device=DEV) + s["pos"]) % q).repeat_interleave(k)
    x = s["X"].float().repeat_interleave(k, 0)
    gate = _project_plain(x, s["Wg"], pair, types, idx, cnt, q, D, F)
    up = _project_plain(x, s["Wu"], pair, types, idx, cnt, q, D, F)
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = _project_plain(h, s["Wd"], pair, types, idx, cnt, q, F, D).view(n, k, D)
    return [(y * weights[..., None]).sum(1).to(DTYPES[s["y"]]), experts.to(torch.int32), weights]


def run(state):
    if own:
        return _run_own(state)
    return {"norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "attn": _attn_plain,
            "moe": _moe_plain}[state["op"]](state)


# --------------------------------------------------------------- definition ---

def _norm_fwd_exact(s):
    x = s["X"].double()
    S = None
    if s["D"] is not None:
        S = (s["X"].double() + s["D"].double()).to(s["X"].dtype)
        x = S.double()
    var, mean = torch.var_mean(x, 1, unbiased=False)
    rstd = (var + EPS).pow(-0.5)
    y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double())
    return [y, None if S is None else S.double(), mean, rstd]


def _norm_bwd_exact(s):
    x, dy = s["X"].double(), s["dY"].double()
    d = x.shape[1]
    var, mean = torch.var_mean(x, 1, unbiased=False)
    xc = x - mean[:, None]
    sd = torch.sqrt(var + EPS)[:, None]
    g = dy * s["gamma"].double()
    # d/dx of (x - mean) / sd with mean and sd as functions of x
    dx = g / sd - g.sum(1, keepdim=True) / (d * sd) - xc * (g * xc).sum(1, keepdim=True) / (d * sd ** 3)
    if s["dS"] is not None:
        dx += s["dS"].double()
    return [dx, torch.matmul(torch.ones(1, x.shape[0], device=DEV, dtype=torch.float64), dy * (xc / sd))[0],
            torch.matmul(torch.ones(1, x.shape[0], device=DEV, dtype=torch.float64), dy)[0]]


def _attn_exact(s):
    B, H, Hkv, D, page = s["B"], s["H"], s["Hkv"], s["D"], s["page"]
    O = torch.zeros(B, H, D, device=DEV, dtype=torch.float64)
    lens, table = s["lens"].tolist(), s["table"]
    rows = s["qkv"].view(B, H + 2 * Hkv, D)
    for b in range(B):
        n = lens[b]
        pg = table[b, (n - 1) // page].item()
        s["Kp"][pg, :, (n - 1) % page] = rows[b, H : H + Hkv].to(torch.bfloat16)
        s["Vp"][pg, :, :, (n - 1) % page] = rows[b, H + Hkv :].to(torch.bfloat16)
    for b in range(B):
        n = lens[b]
        ids = table[b, : -(-n // page)].long()
        for h in range(Hkv):
            K = s["Kp"][ids, h].reshape(-1, D)[:n].double()
            V = s["Vp"][ids, h].transpose(1, 2).reshape(-1, D)[:n].double()
            G = H // Hkv
            for g in range(G):
                a = torch.mv(K, rows[b, h * G + g].double()) / math.sqrt(D)
                O[b, h * G + g] = torch.mv(V.t(), torch.softmax(a, 0))
    return [O, s["Kp"].double(), s["Vp"].double()]


def _dense(W, q, di, do):
    """One expert's packed weight as the di x do matrix, entry by entry from the layout's definition."""
    bi, bo = di // q, do // q
    r = torch.arange(di, device=DEV)[:, None]
    c = torch.arange(do, device=DEV)[None, :]
    kk, nn = r % bi, c % bo
    slab = kk // 32
    at = ((r // bi) * q + c // bo) * (bi * bo) + (nn // 16) * (bi * 16) + slab * 512
    at = at + ((kk % 32) // 8 * 16 + nn % 16) * 8 + kk % 8
    return W[at].double()


def _moe_exact(s):
    n, q, D, F, k, E = s["n"], s["q"], s["D"], s["F"], s["k"], s["E"]
    X, Rt = s["X"].double(), s["R"].double()

    def mask(t, di, do):
        m = torch.zeros(q, q, device=DEV, dtype=torch.float64)
        for j in range(q):
            for o in range(q):
                if s["law"] == "Qq":
                    m[j, o] = float(j == t or j == o)
                else:
                    m[j, o] = float(j >> 1 in (t >> 1, o >> 1) and j & 1 in (t & 1, o & 1))
        return m.repeat_interleave(di // q, 0).repeat_interleave(do // q, 1)

    Y = torch.zeros(n, D, device=DEV, dtype=torch.float64)
    experts, weights = torch.zeros(n, k, dtype=torch.int32), torch.zeros(n, k, dtype=torch.float64)
    for t in range(n):
        logit = [float(v) for v in (X[t] * Rt).sum(1)]
        chosen = sorted(range(E), key=lambda e: (-logit[e], e))[:k]
        top = logit[chosen[0]]
        den = sum(math.exp(logit[e] - top) for e in (chosen if s["norm"] else range(E)))
        tau = (s["pos"] + t) % q
        up, down = mask(tau, D, F), mask(tau, F, D)
        for a, e in enumerate(chosen):
            experts[t, a] = e
            weights[t, a] = math.exp(logit[e] - top) / den
            gate = X[t] @ (_dense(s["Wg"][e], q, D, F) * up)
            h = gate * torch.sigmoid(gate) * (X[t] @ (_dense(s["Wu"][e], q, D, F) * up))
            Y[t] += float(weights[t, a]) * (h @ (_dense(s["Wd"][e], q, F, D) * down))
    return [Y, experts.to(DEV), weights.to(DEV)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_fwd": _norm_fwd_exact, "norm_bwd": _norm_bwd_exact, "attn": _attn_exact,
            "moe": _moe_exact}[s["op"]](s)


# --------------------------------------------------------------------- work ---

def _used_blocks(c):
    """Expected distinct weight blocks of one matrix over all experts, for random routing: a block counts
    where one of the tokens whose type uses it has chosen its expert."""
    q, n = c["q"], c["n"]
    g = np.arange(q)
    i, k, j = g[:, None, None], g[None, :, None], g[None, None, :]
    if c["law"] == "Qq":
        T = (j == i) | (j == k)
    else:
        T = ((j // 2 == i // 2) | (j // 2 == k // 2)) & ((j % 2 == i % 2) | (j % 2 == k % 2))
    per_type = np.bincount((np.arange(n) + c["pos"]) % q, minlength=q)
    tokens = (T * per_type[:, None, None]).sum(0)                     # tokens that use block (k, j)
    distinct = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** tokens).sum()
    products = (T.sum((1, 2)) * per_type).sum() * c["k"]
    return float(distinct), float(products)


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] == "norm_fwd":
        e = size[c["x"]] * (1 if c["delta"] == "none" else 2) + size[c["delta"]] + size[c["y"]]
        return {"bytes": c["M"] * c["d"] * e + 8 * c["d"] + 8 * c["M"], "flops": 9 * c["M"] * c["d"]}
    if c["op"] == "norm_bwd":
        e = size[c["x"]] * (3 if c["ds"] else 2) + size[c["dy"]]
        return {"bytes": c["M"] * c["d"] * e + 12 * c["d"] + 8 * c["M"], "flops": 16 * c["M"] * c["d"]}
    if c["op"] == "attn":
        T = int(_lengths(c).sum())
        B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]
        io = B * D * ((H + 2 * Hkv) * size[c["q"]] + H * size[c["o"]] + 2 * Hkv * 2)
        return {"bytes": 4 * T * Hkv * D + io + 4 * T // c["page"], "flops": 4 * T * H * D}
    distinct, products = _used_blocks(c)
    block = (c["D"] // c["q"]) * (c["F"] // c["q"])
    io = c["n"] * c["D"] * (2 + size[c["y"]]) + 2 * c["E"] * c["D"] + 8 * c["n"] * c["k"]
    return {"bytes": int(3 * distinct * block * 2 + io), "flops": int(6 * products * block + 2 * c["n"] * c["E"] * c["D"])}
