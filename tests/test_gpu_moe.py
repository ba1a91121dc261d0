"""aa_moe_ffn_fwd against the definition: float64 logits and choice, and the
oracle's row-typed projections.  Needs an MI355X.

Tolerance of an output.  u = 2^-24; P(a, B) is the row-typed projection with
the magnitudes |a|, |B|, K the rows that one output sums at most (4 or 2 input
groups).  Gate and up sum K exact products in float32: (K + 8) u P(|x|, |W|).
silu' lies in [-0.1, 1.1], and silu itself is off by (4 + |g|) u (the
exponential's argument and a division), so
  dh = 1.1 dg |up| + |silu| du + (6 + |g|) u |h|,
  dy = P(dh, |Wd|) + (K + 8) u P(|h|, |Wd|)   for each expert,
and a weight is off by (E + 24) u relative (at most E terms of a softmax, the
exponents' rounding u |r - max| <= 24 u here), the sum over the chosen adds
top_k + 4.  Outputs add half a step of their type.
"""
import numpy as np
import pytest
import torch

import aa_inputs as inp
import associative_algebra_block_amd as aa
import oracle
from tests._gpu_util import host, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


class Layer:
    def __init__(self, law, q, D, F, E, seed, out="f32", kind="pos_mod", period=0):
        self.law, self.q, self.D, self.F, self.E = law, q, D, F, E
        self.up = aa.aa_plan_create(law, q, D, F, kind, period, "bf16", "bf16")
        self.down = aa.aa_plan_create(law, q, F, D, kind, period, "bf16", out)
        self.R = inp.gaussian((E, D), seed, D ** -0.5, BF16, DEV)
        self.rm = [inp.gaussian((E, D * F), seed + 1 + i, s ** -0.5, BF16, DEV) for i, s in enumerate((D, D, F))]
        self.W = [torch.empty_like(w) for w in self.rm]
        for plan, rm, w, (a, b) in ((self.up, self.rm[0], self.W[0], (D, F)), (self.up, self.rm[1], self.W[1], (D, F)),
                                    (self.down, self.rm[2], self.W[2], (F, D))):
            for e in range(E):
                aa.aa_pack_weights(plan, rm[e].view(a, b), w[e])

    def run(self, X, k, norm, pos=0, types=None, Y=None, experts=None, weights=None, ws=None, stream=None):
        M = X.shape[0]
        n = aa.aa_moe_ffn_workspace(self.up, self.down, self.E, k, M)
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if ws is None else ws
        Y = torch.full((M, self.D), 77.0, dtype=self.down.out_torch_dtype, device=DEV) if Y is None else Y
        experts = torch.full((M, k), -7, dtype=torch.int32, device=DEV) if experts is None else experts
        weights = torch.full((M, k), 77.0, device=DEV) if weights is None else weights
        aa.aa_moe_ffn_fwd(self.up, self.down, X, self.R, *self.W, Y, k, norm, experts, weights, ws, pos, types, stream)
        return Y, experts, weights

    def check(self, X, k, norm, types, Y, experts, weights):
        X64, R64 = X.double().cpu().numpy(), self.R.double().cpu().numpy()
        K = (4 if self.law == "Q2xQ2" else 2) * max(self.D, self.F) // self.q
        rows = {}
        for t in range(X.shape[0]):
            r = (X64[t] * R64).sum(1)
            sel = sorted(range(self.E), key=lambda e: (-r[e], e))[:k]
            assert experts[t].tolist() == sel, (t, experts[t].tolist(), sel)
            ex = np.exp(r - r.max())
            w = ex[sel] / (ex[sel].sum() if norm else ex.sum())
            assert np.all(np.abs(weights[t].double().cpu().numpy() - w) <= (self.E + 24) * U * w)
            for e, we in zip(sel, w):
                rows.setdefault(e, []).append((t, we))
        ref, tol = np.zeros((X.shape[0], self.D)), np.zeros((X.shape[0], self.D))
        mag = np.zeros_like(ref)
        for e, tw in rows.items():
            ts, we = [t for t, _ in tw], np.array([w for _, w in tw])[:, None]
            ty = np.asarray(types)[ts]
            Wg, Wu, Wd = (host(m[e]).astype(np.float64).reshape(s) for m, s in
                          zip(self.rm, ((self.D, self.F), (self.D, self.F), (self.F, self.D))))
            x = X64[ts]
            P = lambda a, B: oracle.project(a, B, self.law, self.q, ty)
            g, u = P(x, Wg), P(x, Wu)
            dg, du = ((K + 8) * U * P(np.abs(x), np.abs(W)) for W in (Wg, Wu))
            s = oracle.silu(g)
            h = s * u
            dh = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + (6 + np.abs(g)) * U * np.abs(h)
            y = P(h, Wd)
            ref[ts] += we * y
            tol[ts] += we * (P(dh, np.abs(Wd)) + (K + 8) * U * P(np.abs(h), np.abs(Wd)))
            mag[ts] += we * np.abs(y)
        tol += (self.E + 24 + k + 4) * U * mag
        tol += torch.finfo(Y.dtype).eps / 2 * (np.abs(ref) + tol)
        err = np.abs(Y.double().cpu().numpy() - ref)
        say(f"moe: worst error / bound {float((err / np.maximum(tol, 1e-300)).max()):.3f}")
        assert np.all(err <= tol), float((err - tol).max())


CASES = [  # law, q, D, F, E, top_k, M, normalize, out, pos
    ("Qq", 16, 2048, 768, 12, 8, 3, True, "bf16", 37),       # the expert FFN; 48-wide blocks (half slabs) in the down products
    ("Qq", 16, 2048, 768, 4, 2, 20, True, "f32", 5),         # every type, and more than one token a type
    ("Q2xQ2", 4, 768, 1536, 8, 2, 5, False, "f32", 6),
    ("Q2xQ2", 4, 64, 192, 3, 3, 7, False, "f32", 1),
    ("Qq", 1, 64, 48, 6, 5, 2, True, "f32", 0),              # q = 1 is the plain FFN; top_k no multiple of 4
    ("Qq", 2, 96, 32, 1, 1, 3, True, "f32", 9),              # one expert
    ("Qq", 3, 144, 240, 5, 4, 4, False, "bf16", 2),          # 48- and 80-wide blocks
    ("Qq", 4, 64, 64, 512, 64, 2, False, "f32", 3),          # the limits
    ("Qq", 4, 64, 64, 300, 7, 3, True, "f32", 3),
    ("Qq", 2, 1024, 2080, 3, 2, 2, True, "f32", 1),          # wide blocks: several rounds of loads
    ("Qq", 8, 128, 128, 9, 1, 33, False, "f32", 100),
    ("Qq", 4, 64, 320, 6, 3, 30, True, "f32", 1),            # 90 pairs in rows of eight, three workgroups each
    ("Qq", 2, 64, 160, 6, 3, 30, False, "bf16", 0),
]


@pytest.mark.parametrize("law,q,D,F,E,k,M,norm,out,pos", CASES)
def test_layer(law, q, D, F, E, k, M, norm, out, pos):
    say("moe", law, q, D, F, E, k, M, norm, out, pos)
    L = Layer(law, q, D, F, E, 40 + D + E, out)
    X = inp.gaussian((M, D), 7 + M, 1.0, BF16, DEV)
    Y, experts, weights = L.run(X, k, norm, pos)
    torch.cuda.synchronize()
    L.check(X, k, norm, oracle.types_pos_mod(M, q, pos), Y, experts, weights)


# the kernels that the sizes above do not reach: long sums of few strips (eight waves a strip), two strips a
# workgroup of eight waves, and of either width with a strip left over (an odd number of them in an output group)
KERNEL_CASES = [
    ("Q2xQ2", 4, 768, 1536, 8, 2, 1, True, "f32", 3),
    ("Q2xQ2", 4, 768, 1536, 8, 2, 1, False, "bf16", 6),
    ("Q2xQ2", 4, 768, 1536, 8, 2, 20, True, "f32", 1),
    ("Q2xQ2", 4, 768, 1536, 8, 2, 20, False, "bf16", 2),
    ("Qq", 2, 640, 1440, 15, 6, 7, True, "f32", 0),
    ("Qq", 4, 192, 64, 5, 2, 34, True, "f32", 3),
    ("Qq", 4, 192, 64, 5, 3, 35, False, "bf16", 1),
    ("Qq", 4, 192, 64, 5, 2, 130, True, "f32", 2),
    ("Qq", 4, 192, 64, 5, 2, 131, False, "bf16", 0),
    ("Qq", 1, 80, 48, 4, 2, 90, True, "f32", 0),
    ("Qq", 4, 128, 64, 4, 2, 400, False, "bf16", 2),
    ("Qq", 4, 128, 64, 4, 2, 400, True, "f32", 2),
]


@pytest.mark.parametrize("law,q,D,F,E,k,M,norm,out,pos", KERNEL_CASES)
def test_layer_on_every_kernel(law, q, D, F, E, k, M, norm, out, pos):
    test_layer(law, q, D, F, E, k, M, norm, out, pos)


def test_equal_logits_go_to_the_lower_index():
    L = Layer("Qq", 2, 64, 64, 70, 3)
    L.R[5], L.R[69], L.R[64] = L.R[33], L.R[33], L.R[33]
    L.R[10:20] = 0
    X = inp.gaussian((6, 64), 5, 1.0, BF16, DEV)
    X[0] = L.R[33] * 50                      # 5, 33, 64 and 69 lead
    X[1] = 0                                 # all equal
    Y, experts, weights = L.run(X, 6, True)
    assert experts[0, :4].tolist() == [5, 33, 64, 69] and experts[1].tolist() == [0, 1, 2, 3, 4, 5]
    assert torch.equal(weights[1], torch.full((6,), 1.0, device=DEV) / 6)
    L.check(X, 6, True, oracle.types_pos_mod(6, 2, 0), Y, experts, weights)


def test_sequences_end_to_end_and_large_positions():
    L = Layer("Qq", 4, 64, 64, 5, 11, period=8)
    X = inp.gaussian((19, 64), 5, 1.0, BF16, DEV)
    out = L.run(X, 2, True, 6)
    L.check(X, 2, True, oracle.types_pos_mod(19, 4, 6, 8), *out)
    P = Layer("Qq", 3, 48, 48, 5, 11)
    X = inp.gaussian((4, 48), 5, 1.0, BF16, DEV)
    pos = (1 << 62) + 1
    out = P.run(X, 2, True, pos)
    P.check(X, 2, True, [(pos + t) % 3 for t in range(4)], *out)


def test_explicit_types_and_rows_left_alone():
    L = Layer("Q2xQ2", 4, 64, 128, 6, 13, "bf16", "explicit")
    X = inp.gaussian((7, 64), 5, 1.0, BF16, DEV)
    types = torch.tensor([3, -1, 0, 4, 2, 1 << 30, 1], dtype=torch.int32, device=DEV)
    Y, experts, weights = L.run(X, 3, True, types=types)
    torch.cuda.synchronize()
    skipped, kept = [1, 3, 5], [0, 2, 4, 6]
    assert bool((Y[skipped] == 77).all()) and bool((experts[skipped] == -7).all()) and bool((weights[skipped] == 77).all())
    L.check(X[kept], 3, True, types[kept].cpu().numpy(), Y[kept], experts[kept], weights[kept])


@pytest.mark.parametrize("law,q,E,k", [("Qq", 2, 8, 3), ("Q2xQ2", 4, 70, 5)])
@pytest.mark.parametrize("x_exp,r_exp", [(-80, -60), (-63, -66), (80, 60), (64, 63), (-100, -50)])
def test_choice_where_float32_has_no_such_products(law, q, E, k, x_exp, r_exp):
    """Logits are float64: scaling the token and the router by powers of two
    scales them exactly, also where a float32 product would be infinite, zero or
    short of digits.  (The experts' own float32 sums need not hold such values;
    weights are those of the logits' differences.)"""
    say("moe choice", law, q, E, k, x_exp, r_exp)
    L = Layer(law, q, 64, 64, E, 37)
    X = inp.gaussian((6, 64), 5, 1.0, BF16, DEV)
    base = (X.double() @ L.R.double().t()).cpu().numpy()
    X = (X.double() * 2.0 ** x_exp).to(BF16)
    L.R = (L.R.double() * 2.0 ** r_exp).to(BF16)
    assert torch.equal((X.double() @ L.R.double().t()).cpu(), torch.from_numpy(base * 2.0 ** (x_exp + r_exp)))
    for norm in (True, False):
        _, experts, weights = L.run(X, k, norm)
        r = base * 2.0 ** (x_exp + r_exp)
        for t in range(6):
            sel = sorted(range(E), key=lambda e: (-r[t, e], e))[:k]
            assert experts[t].tolist() == sel, (t, experts[t].tolist(), sel)
            ex = np.exp(r[t] - r[t].max())
            w = ex[sel] / (ex[sel].sum() if norm else ex.sum())
            # a weight below float32's normal values is off by half its smallest step
            assert np.all(np.abs(weights[t].double().cpu().numpy() - w) <= (E + 24) * U * w + 2.0 ** -150)


def test_a_token_of_nan_stays_alone():
    L = Layer("Qq", 2, 64, 64, 8, 17)
    X = inp.gaussian((5, 64), 5, 1.0, BF16, DEV)
    good = [t.clone() for t in L.run(X, 2, False)]
    X[2, 7] = float("nan")
    bad = L.run(X, 2, False)
    rest = [0, 1, 3, 4]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(good, bad))
    assert bool(bad[0][2].isnan().all()) and bool(bad[2][2].isnan().all())
    assert bad[1][2].tolist() == [0, 1]


def test_the_most_pairs_equal_parts_of_them():
    """65535 (token, expert) pairs in one call give what 15 calls give; the last
    tokens also against the definition."""
    L = Layer("Qq", 2, 64, 32, 3, 19)
    M, part = 65535, 4369
    X = inp.gaussian((M, 64), 5, 1.0, BF16, DEV)
    all_at_once = L.run(X, 1, False, 1)
    parts = [L.run(X[lo:lo + part], 1, False, 1 + lo) for lo in range(0, M, part)]
    for i, t in enumerate(all_at_once):
        assert torch.equal(t, torch.cat([p[i] for p in parts]))
    last = slice(M - 9, M)
    L.check(X[last], 1, False, oracle.types_pos_mod(9, 2, 1 + M - 9), *(t[last] for t in all_at_once))


def test_one_expert_is_the_ffn():
    """One expert with weight one is aa_swiglu_ffn_fwd, which rounds the hidden
    activation to bf16 (2^-9 of each, in quadrature well below 2^-8 of y)."""
    L = Layer("Qq", 16, 512, 768, 1, 19)
    X = inp.gaussian((3, 512), 5, 1.0, BF16, DEV)
    Y, experts, weights = L.run(X, 1, True, 4)
    ref, H = torch.empty_like(Y), torch.empty(3, 768, dtype=BF16, device=DEV)
    aa.aa_swiglu_ffn_fwd(L.up, L.down, X, L.W[0][0], L.W[1][0], L.W[2][0], H, ref, None, 4)
    assert bool((weights == 1).all()) and bool((experts == 0).all())
    assert float((Y - ref).norm() / ref.norm()) < 2.0 ** -8


def test_offsets_beyond_32_bits():
    """512 experts of 2048 x 2304: more than 2^31 elements a matrix; the last
    expert is chosen."""
    q, D, F, E = 16, 2048, 2304, 512
    L = Layer.__new__(Layer)
    L.law, L.q, L.D, L.F, L.E = "Qq", q, D, F, E
    L.up = aa.aa_plan_create("Qq", q, D, F, "pos_mod", 0, "bf16", "bf16")
    L.down = aa.aa_plan_create("Qq", q, F, D, "pos_mod", 0, "bf16", "f32")
    L.R = torch.zeros(E, D, dtype=BF16, device=DEV)
    X = inp.gaussian((2, D), 5, 1.0, BF16, DEV)
    L.R[511], L.R[510] = X[0] / 16, X[1] / 16
    small = [inp.gaussian((2, D * F), 60 + i, s ** -0.5, BF16, DEV) for i, s in enumerate((D, D, F))]
    L.W = [torch.empty(E, D * F, dtype=BF16, device=DEV) for _ in range(3)]
    for i, (plan, a, b) in enumerate(((L.up, D, F), (L.up, D, F), (L.down, F, D))):
        for e in range(2):
            aa.aa_pack_weights(plan, small[i][e].view(a, b), L.W[i][510 + e])
    out = L.run(X, 1, True, 3)
    assert out[1].tolist() == [[511], [510]]

    class Last:
        def __init__(self, t):
            self.t = t

        def __getitem__(self, e):
            return self.t[e - 510]

    L.rm = [Last(t) for t in small]
    L.check(X, 1, True, oracle.types_pos_mod(2, q, 3), *out)


def test_repeats_streams_and_graphs():
    """Two captured layers of different sizes share a workspace; replays between
    eager calls on changing inputs equal the eager results bit for bit."""
    a, b = Layer("Qq", 16, 512, 768, 10, 23), Layer("Q2xQ2", 4, 128, 64, 5, 29, "bf16")
    Xa, Xb = inp.gaussian((4, 512), 5, 1.0, BF16, DEV), inp.gaussian((2, 128), 6, 1.0, BF16, DEV)
    ws = torch.empty(max(aa.aa_moe_ffn_workspace(a.up, a.down, 10, 4, 4), aa.aa_moe_ffn_workspace(b.up, b.down, 5, 2, 2)),
                     dtype=torch.uint8, device=DEV)
    outa, outb = a.run(Xa, 4, True, 1, ws=ws), b.run(Xb, 2, False, 1, ws=ws)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a.run(Xa, 4, True, 1, None, *outa, ws=ws)
    with torch.cuda.graph(gb):
        b.run(Xb, 2, False, 1, None, *outb, ws=ws)
    side = torch.cuda.Stream()
    for r in range(4):
        Xa.normal_()
        Xb.normal_()
        wa, wb = a.run(Xa, 4, True, 1, ws=ws), b.run(Xb, 2, False, 1, ws=ws)
        ga.replay()
        gb.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outa + outb, wa + wb)), r
        with torch.cuda.stream(side):
            wa2 = a.run(Xa, 4, True, 1)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(wa, wa2))


def test_no_tokens_and_optional_outputs():
    L = Layer("Qq", 2, 64, 64, 4, 31)
    L.run(torch.empty(0, 64, dtype=BF16, device=DEV), 2, True)
    X = inp.gaussian((2, 64), 5, 1.0, BF16, DEV)
    Y, _, _ = L.run(X, 2, True)
    Z = torch.empty_like(Y)
    ws = torch.empty(aa.aa_moe_ffn_workspace(L.up, L.down, 4, 2, 2), dtype=torch.uint8, device=DEV)
    aa.aa_moe_ffn_fwd(L.up, L.down, X, L.R, *L.W, Z, 2, True, workspace=ws)
    assert torch.equal(Y, Z)


def test_binding_refuses_before_the_library():
    L = Layer("Qq", 2, 64, 64, 4, 31)
    X, Y = inp.gaussian((2, 64), 5, 1.0, BF16, DEV), torch.empty(2, 64, device=DEV)
    ws = torch.empty(aa.aa_moe_ffn_workspace(L.up, L.down, 4, 2, 2), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="shape"):
        aa.aa_moe_ffn_fwd(L.up, L.down, X, L.R, L.W[0][:3], L.W[1], L.W[2], Y, 2, workspace=ws)
    with pytest.raises(TypeError, match="dtype"):
        aa.aa_moe_ffn_fwd(L.up, L.down, X, L.R, *L.W, Y.to(BF16), 2, workspace=ws)
    with pytest.raises(TypeError, match="dtype"):
        aa.aa_moe_ffn_fwd(L.up, L.down, X, L.R.float(), *L.W, Y, 2, workspace=ws)
    with pytest.raises(aa.AAError, match="top_k exceeds"):
        aa.aa_moe_ffn_fwd(L.up, L.down, X, L.R, *L.W, Y, 5, workspace=ws)
    with pytest.raises(aa.AAError, match="workspace"):
        aa.aa_moe_ffn_fwd(L.up, L.down, X, L.R, *L.W, Y, 2)
