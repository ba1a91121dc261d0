"""LayerNorm, paged attention and the mixture-of-experts layer in one run, as a
decoder calls them: decode steps of a block with an MoE feed-forward, and a
training step of a norm and a row-typed projection.  Needs an MI355X.

The references are float64 and round to bf16 where the run stores bf16 (the
norms' outputs, keys and values, the attention's output).  A rounding that
falls on the other side there moves one value by 2^-8 of itself, which is what
the bound on the block's output allows in the Frobenius norm (2^-8, while all
but a few values agree to float32)."""
import math

import numpy as np
import pytest
import torch

import aa_inputs as inp
import associative_algebra_block_amd as aa
import oracle
from tests._gpu_util import metrics, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def bf(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(BF16).double().numpy()


def h64(t):
    return t.double().cpu().numpy()


def ln(x, w, b):
    mu = x.mean(-1, keepdims=True)
    return (x - mu) / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + EPS) * w + b


def test_decode_steps_of_a_block_with_experts():
    """Three sequences (one joins at the second step, one leaves) over six
    steps across a page's end: residual norms, append, attention, norm, MoE."""
    B, H, Hkv, hd, page, steps = 3, 8, 2, 32, 16, 6
    D, F, E, k, q = H * hd, 512, 6, 2, 4
    W = (H + 2 * Hkv) * hd
    Wqkv, Wo = inp.gaussian((D, W), 1, D ** -0.5, BF16, DEV), inp.gaussian((D, D), 2, D ** -0.5, BF16, DEV)
    g1, b1, g2, b2 = (inp.gaussian((D,), s, 0.1, F32, DEV) + o for s, o in ((3, 1), (4, 0), (5, 1), (6, 0)))
    R = inp.gaussian((E, D), 7, D ** -0.5, BF16, DEV)
    up = aa.aa_plan_create("Qq", q, D, F, "explicit", 0, "bf16", "bf16")
    down = aa.aa_plan_create("Qq", q, F, D, "explicit", 0, "bf16", "f32")
    rm = [inp.gaussian((E, D * F), 8 + i, s ** -0.5, BF16, DEV) for i, s in enumerate((D, D, F))]
    packed = [torch.empty_like(w) for w in rm]
    for e in range(E):
        for plan, w, p, sh in ((up, rm[0], packed[0], (D, F)), (up, rm[1], packed[1], (D, F)), (down, rm[2], packed[2], (F, D))):
            aa.aa_pack_weights(plan, w[e].view(sh), p[e])
    table = torch.tensor([[4, 0], [1, 5], [3, 2]], dtype=torch.int32, device=DEV)
    Kp = torch.full((6, Hkv, page, hd), float("nan"), dtype=BF16, device=DEV)
    Vp = torch.full((6, Hkv, hd, page), float("nan"), dtype=BF16, device=DEV)
    start = [13, 0, 2]                                   # positions already in the cache
    past = [[np.zeros((0, Hkv, hd)), np.zeros((0, Hkv, hd))] for _ in range(B)]
    for s, n in enumerate(start):
        if n:
            rows = inp.gaussian((n, 2 * Hkv * hd), 20 + s, 1.0, F32, DEV)
            aa.aa_kv_append(rows[:, :Hkv * hd], rows[:, Hkv * hd:], Kp, Vp, table,
                            torch.arange(n, dtype=torch.int32, device=DEV),
                            torch.full((n,), s, dtype=torch.int32, device=DEV))
            past[s] = [bf(h64(rows[:, :Hkv * hd])).reshape(n, Hkv, hd), bf(h64(rows[:, Hkv * hd:])).reshape(n, Hkv, hd)]
    ws_attn = torch.empty(max(aa.aa_attn_decode_workspace(B, H, Hkv, hd, page, 2), 16), dtype=torch.uint8, device=DEV)
    ws_moe = torch.empty(aa.aa_moe_ffn_workspace(up, down, E, k, B), dtype=torch.uint8, device=DEV)
    n = list(start)
    for step in range(steps):
        live = [True, step >= 1, step < 4]
        pos = torch.tensor([n[s] if live[s] else -1 for s in range(B)], dtype=torch.int32, device=DEV)
        lens = pos + 1                                   # a sequence that sits out attends to nothing
        types = torch.where(pos >= 0, pos % q, -1).to(torch.int32)
        x = inp.gaussian((B, D), 100 + step, 1.0, F32, DEV)
        x0 = h64(x)
        a, f, o = (torch.empty(B, D, dtype=BF16, device=DEV) for _ in range(3))
        aa.aa_layernorm_fwd(x, g1, b1, a)
        qkv = torch.matmul(a, Wqkv).float()
        aa.aa_kv_append(qkv[:, D:D + Hkv * hd], qkv[:, D + Hkv * hd:], Kp, Vp, table, pos)
        aa.aa_attn_decode(qkv[:, :D], Kp, Vp, table, lens, o.view(B, H, hd), hd ** -0.5, ws_attn)
        att = torch.matmul(o, Wo)
        aa.aa_layernorm_fwd(x, g2, b2, f, att, x)
        y = torch.zeros(B, D, device=DEV)
        aa.aa_moe_ffn_fwd(up, down, f, R, *packed, y, k, True, workspace=ws_moe, row_types=types)
        out = (x + y).double().cpu().numpy()
        torch.cuda.synchronize()

        # the same from the definitions, each part on the run's own stored inputs
        qv = h64(qkv).reshape(B, H + 2 * Hkv, hd)
        ra = ln(x0, h64(g1), h64(b1))
        assert metrics(h64(a), ra)[0] <= 2.0 ** -8
        for s in range(B):
            if not live[s]:
                assert bool((o[s] == 0).all()) and np.array_equal(out[s], h64(x)[s])
                continue
            for i, part in enumerate((qv[s, H:H + Hkv], qv[s, H + Hkv:])):
                past[s][i] = np.concatenate([past[s][i], bf(part)[None]])
            K, V = past[s]
            ro = np.zeros((H, hd))
            for hh in range(H):
                sc = K[:, hh // (H // Hkv)] @ qv[s, hh] / math.sqrt(hd)
                p = np.exp(sc - sc.max())
                ro[hh] = p @ V[:, hh // (H // Hkv)] / p.sum()
            assert metrics(h64(o[s]), ro.reshape(-1))[0] <= 2.0 ** -8, (step, s)
            r = h64(f)[s] @ h64(R).T
            sel = sorted(range(E), key=lambda e: (-r[e], e))[:k]
            w = np.exp(r[sel] - r[sel].max())
            w /= w.sum()
            ref = np.zeros(D)
            for e, we in zip(sel, w):
                Wg, Wu, Wd = (h64(m[e]).reshape(sh) for m, sh in zip(rm, ((D, F), (D, F), (F, D))))
                ty = np.array([n[s] % q])
                P = lambda v, M: oracle.project(v, M, "Qq", q, ty)
                ref += we * P(oracle.silu(P(h64(f)[s:s + 1], Wg)) * P(h64(f)[s:s + 1], Wu), Wd)[0]
            assert metrics(h64(y[s]), ref)[0] <= 1e-5, (step, s)
            # the whole block from its input
            x1 = x0[s] + bf(bf(ro.reshape(-1)) @ h64(Wo))
            assert metrics(h64(f[s]), ln(x1, h64(g2), h64(b2)))[0] <= 2.0 ** -7, (step, s)
            assert metrics(out[s], x1 + ref)[0] <= 2.0 ** -8, (step, s)
            n[s] += 1
    say(f"block with experts: {steps} steps, lengths {n}")


@pytest.mark.parametrize("M,D,F,q", [(96, 256, 512, 4), (33, 128, 384, 2)])
def test_training_step_of_norm_and_projection(M, D, F, q):
    """s = x + delta, a = norm(s), z = a * W and a loss linear in z and s: the
    gradients of x, delta, gamma, beta and W against float64 autograd through
    the closed form of the product (a is rounded to bf16 in both, and its
    gradient passes the rounding as it is).  Bound: float32 sums of at most 1024
    terms, 2^-14 relative to what is summed, in the Frobenius norm."""
    x, delta = inp.gaussian((M, D), 1, 1.0, F32, DEV), inp.gaussian((M, D), 2, 0.5, BF16, DEV)
    gamma, beta = inp.gaussian((D,), 3, 0.2, F32, DEV) + 1, inp.gaussian((D,), 4, 0.2, F32, DEV)
    Wm = inp.gaussian((D, F), 5, D ** -0.5, BF16, DEV)
    dz, ds = inp.gaussian((M, F), 6, 1.0, BF16, DEV), inp.gaussian((M, D), 7, 1.0, F32, DEV)
    plan = aa.aa_plan_create("Qq", q, D, F, "pos_mod", 0, "bf16", "f32")
    s, a = torch.empty_like(x), torch.empty(M, D, dtype=BF16, device=DEV)
    mean, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    aa.aa_layernorm_fwd(x, gamma, beta, a, delta, s, mean, rstd, EPS)
    Wp = aa.pack(plan, Wm)
    z = aa.project(plan, a, Wp, 3)
    nd, nw = aa.aa_project_bwd_workspace(plan, M)
    wsd, wsw = (torch.empty(max(n, 16), dtype=torch.uint8, device=DEV) for n in (nd, nw))
    da, dWp = torch.empty(M, D, device=DEV), torch.empty(D * F, device=DEV)
    aa.aa_project_bwd_data(plan, dz, Wp, da, None, 3, None, wsd, nd)
    aa.aa_project_bwd_weight(plan, a, dz, dWp, None, 3, None, wsw, nw)
    dgamma, dbeta = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(aa.aa_layernorm_bwd_workspace(M, D), dtype=torch.uint8, device=DEV)
    aa.aa_layernorm_bwd(s, da, gamma, mean, rstd, ds_out := ds.clone(), dgamma, dbeta, ds_out, ws)
    dW = torch.empty(D, F, device=DEV)
    aa.aa_unpack_weights(aa.aa_plan_create("Qq", q, D, F, "pos_mod", 0, "f32", "f32"), dWp, dW)
    torch.cuda.synchronize()

    X, Dl, G, Bt, W64 = (t.double().cpu().requires_grad_() for t in (x, delta, gamma, beta, Wm))
    S = X + Dl
    A = torch.nn.functional.layer_norm(S, (D,), G, Bt, EPS)
    Aq = A + (A.detach().to(BF16).double() - A.detach())
    bi, bo = D // q, F // q
    blocks = W64.view(q, bi, q, bo)
    off = blocks * (1 - torch.eye(q, dtype=torch.float64))[:, None, :, None]
    keep = torch.ones(M, q, dtype=torch.float64)
    keep[torch.arange(M), (torch.arange(M) + 3) % q] = 0          # all groups but the row's own
    Z = Aq @ W64 - (Aq.view(M, q, bi) * keep[..., None]).reshape(M, D) @ off.reshape(D, F)
    ((Z * dz.double().cpu()).sum() + (S * ds.double().cpu()).sum()).backward()
    for name, got, ref in (("z", z, Z.detach()), ("dx", ds_out, X.grad), ("ddelta", ds_out, Dl.grad),
                           ("dgamma", dgamma, G.grad), ("dbeta", dbeta, Bt.grad), ("dW", dW, W64.grad)):
        rel, _ = metrics(h64(got), ref.numpy())
        say(f"training step {M} x {D} -> {F}: {name} {rel:.2e}")
        # a rounding of a that falls on the other side shows in z and dW
        assert rel <= (2.0 ** -12 if name in ("z", "dW") else 2.0 ** -14), (name, rel)
