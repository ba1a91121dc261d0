"""aa_attn_decode and aa_kv_append against the definitions in float64.  Needs
an MI355X.

Tolerance of an output element.  u = 2^-24.  A score sums D products of bf16
terms (3 D for float32 queries) in float32: it is off by at most
n u sum |scale q k| with n = 3 D + 3 (the scale and the product's rounding),
so its probability by the factor exp of that; the exponential's argument and
result add 8 u (1 + max |s - m|).  Two bf16 terms of a probability leave
2^-17 of it (float32 outputs take three: 2^-25).  The weighted sum over len
positions and its denominator add 2 (len / 8 + 64) u: at most len / 32 steps of
a wave, each adding at most 4 roundings, 4 waves, 256 splits joined in order.
So |err| <= (2 eps_s + eps_p + eps_sum) sum p |v|, plus half a step of the
output's type.
"""
import math

import pytest
import torch

import associative_algebra_block_amd as aa
from tests._gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


class Cache:
    """Pages in a seeded random order, filled with `fill`, and a table whose
    unused entries point nowhere."""

    def __init__(self, lens, Hkv, D, page, seed, fill=float("nan"), cap=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        self.most = max(max(need), 1) if cap is None else cap
        n_pages = sum(need) + 2
        order = torch.randperm(n_pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), self.most), 1 << 30, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            table[b, k:] = -1 if b % 2 else 1 << 30
            at += k
        self.table = table.to(DEV)
        self.K = torch.full((n_pages, Hkv, page, D), fill, dtype=BF16, device=DEV)
        self.V = torch.full((n_pages, Hkv, D, page), fill, dtype=BF16, device=DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.k = [torch.randn(max(n, 0), Hkv, D, generator=g).to(BF16).to(DEV) for n in lens]
        self.v = [torch.randn(max(n, 0), Hkv, D, generator=g).to(BF16).to(DEV) for n in lens]
        self.page, self.Hkv, self.D = page, Hkv, D

    def write(self):
        """Put every position in its slot with plain indexing."""
        for b, (k, v) in enumerate(zip(self.k, self.v)):
            for lo in range(0, k.shape[0], self.page):
                pg = int(self.table[b, lo // self.page])
                n = min(self.page, k.shape[0] - lo)
                self.K[pg, :, :n] = k[lo:lo + n].transpose(0, 1)
                self.V[pg, :, :, :n] = v[lo:lo + n].permute(1, 2, 0)
        return self

    def workspace(self, H):
        n = aa.aa_attn_decode_workspace(len(self.k), H, self.Hkv, self.D, self.page, self.most)
        return torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)


def attend(c, Q, o_dtype, scale, H, ws=None, lens=None, stream=None):
    B = len(c.k)
    buf = torch.full((B * H * c.D + 128,), 77.0, dtype=o_dtype, device=DEV)
    O = buf[64:-64].view(B, H, c.D)
    aa.aa_attn_decode(Q, c.K, c.V, c.table, c.lens if lens is None else lens, O, scale,
                      c.workspace(H) if ws is None else ws, stream)
    torch.cuda.synchronize()
    assert bool((buf[:64] == 77.0).all()) and bool((buf[-64:] == 77.0).all())
    return O


def check(c, Q, O, scale, H):
    B, G, D = len(c.k), H // c.Hkv, c.D
    q = Q.reshape(B, H, D).double().cpu()
    worst = 0.0
    half = torch.finfo(O.dtype).eps / 2
    for b in range(B):
        got = O[b].double().cpu()
        n = c.k[b].shape[0]
        if n == 0:
            assert bool((got == 0).all()), b
            continue
        k = c.k[b].double().cpu().repeat_interleave(G, 1)                 # [n, H, D]
        v = c.v[b].double().cpu().repeat_interleave(G, 1)
        s = (k * q[b]).sum(2) * scale                                     # [n, H]
        p = torch.softmax(s, 0)
        ref = (p[..., None] * v).sum(0)
        mag = (k * q[b]).abs().sum(2).max(0).values * abs(scale)
        spread = (s.max(0).values - s.min(0).values)
        eps_s = (3 * D + 3) * U * mag + 8 * U * (1 + spread)
        eps_p = 2.0 ** -17 if O.dtype == BF16 else 2.0 ** -25
        tol = (2 * eps_s + eps_p + 2 * (n / 8 + 64) * U)[:, None] * (p[..., None] * v.abs()).sum(0)
        tol = tol + half * (ref.abs() + tol)
        err = (got - ref).abs()
        worst = max(worst, float((err / tol).max()))
        assert bool((err <= tol).all()), (b, n, worst)
    say(f"attention: worst error / bound {worst:.3f}")


def queries(B, H, D, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, H * D, generator=g) * std).to(dtype).to(DEV)


LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 0, 255, 256, 257, 700]


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 24), (2, 1, 8), (6, 2, 64), (3, 3, 128), (8, 1, 40)])
@pytest.mark.parametrize("qt,ot", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
def test_ragged_batch(page, H, Hkv, D, qt, ot):
    """Lengths around every border, two of them zero; slots behind the ends
    hold NaN."""
    say("attention ragged", page, H, Hkv, D, qt, ot)
    c = Cache(LENS, Hkv, D, page, 100 + page + D).write()
    Q = queries(len(LENS), H, D, qt, D)
    check(c, Q, attend(c, Q, ot, D ** -0.5, H), D ** -0.5, H)


@pytest.mark.parametrize("D", [16, 32, 48, 72, 80, 96, 104, 136, 160, 184, 192, 216, 224, 248, 256])
def test_head_dims(D):
    say("attention head dim", D)
    c = Cache([1, 40, 333], 2, D, 64, D).write()
    for qt, ot in ((F32, F32), (BF16, BF16)):
        Q = queries(3, 4, D, qt, D)
        check(c, Q, attend(c, Q, ot, D ** -0.5, 4), D ** -0.5, 4)


@pytest.mark.parametrize("H,Hkv", [(16, 1), (17, 1), (20, 1), (33, 1), (40, 2), (15, 5)])
def test_head_groups(H, Hkv):
    """More than 16 query heads of a kv head: several tiles of heads."""
    say("attention groups", H, Hkv)
    c = Cache([5, 129, 0, 900], Hkv, 32, 32, H).write()
    Q = queries(4, H, 32, BF16, H)
    check(c, Q, attend(c, Q, F32, 0.2, H), 0.2, H)


@pytest.mark.parametrize("lens,cap", [([5000], None), ([40000, 3], None), ([257, 8191, 1, 0], None), ([300], 4096)])
def test_long_sequences_are_split_and_joined(lens, cap):
    say("attention long", lens, cap)
    H, Hkv, D = 4, 2, 64
    c = Cache(lens, Hkv, D, 16 if cap else 64, sum(lens), cap=cap).write()
    assert aa.aa_attn_decode_workspace(len(lens), H, Hkv, D, c.page, c.most) > 0
    Q = queries(len(lens), H, D, F32, 7, 2.0)
    check(c, Q, attend(c, Q, F32, D ** -0.5, H), D ** -0.5, H)


def test_sharp_and_large_scores():
    """Scores in the hundreds, growing and falling along the sequence: the
    running maximum moves in every step."""
    c = Cache([600, 600], 1, 32, 32, 3)
    ramp = torch.linspace(-4, 4, 600, device=DEV)
    c.k[0] = (ramp[:, None, None] * torch.ones(1, 1, 32, device=DEV)).to(BF16)
    c.k[1] = c.k[0].flip(0).contiguous()
    c.write()
    Q = torch.full((2, 2 * 32), 3.0, device=DEV)
    check(c, Q, attend(c, Q, F32, 1.0, 2), 1.0, 2)


def test_infinities_and_nan_follow_the_formula():
    """A key that makes a score -inf has weight 0; a sequence whose scores are
    all -inf, and one with a NaN key, give NaN; the others stay as they are."""
    c = Cache([300, 40, 70, 50], 1, 24, 16, 5)
    for b in range(4):
        c.k[b] = c.k[b].abs()
    c.k[0][17, 0, 3] = float("-inf")
    c.k[1][:, 0, 0] = float("-inf")
    c.k[2][69, 0, 5] = float("nan")
    c.write()
    Q = queries(4, 2, 24, F32, 9).abs() + 0.1
    O = attend(c, Q, F32, 0.3, 2)
    assert bool(O[1].isnan().all()) and bool(O[2].isnan().all())
    keep = [i for i in range(300) if i != 17]
    c.k[0], c.v[0] = c.k[0][keep], c.v[0][keep]
    c.k[1], c.v[1] = c.k[1][:0], c.v[1][:0]
    c.k[2], c.v[2] = c.k[2][:0], c.v[2][:0]
    O[1:3] = 0
    check(c, Q, O, 0.3, 2)


@pytest.mark.parametrize("ot", [F32, BF16])
@pytest.mark.parametrize("D", [8, 40, 160])
def test_queries_beyond_the_largest_bf16_value(D, ot):
    """float32 queries up to float32's largest value, which a rounding to bf16
    would make infinite, against keys so small that the scores are of order
    one; infinite and NaN queries give NaN."""
    top = torch.finfo(F32).max
    c = Cache([70, 700, 5, 9], 1, D, 16, 50 + D)
    for k in c.k:                                             # no denormal values
        k.copy_((torch.sign(k.float()) * (1 + k.float().abs().remainder(1)) * 2.0 ** -124).to(BF16))
    c.write()
    Q = torch.zeros(4, 2, D)
    Q[0, 0, 3], Q[0, 1, 2] = top, -top
    Q[1, 0, 0], Q[1, 0, 7], Q[1, 1, 5] = -top, top * (1 - 2.0 ** -9), top * (1 - 2.0 ** -10)
    Q[2, 0, 4], Q[2, 1, 4] = torch.finfo(BF16).max, top * 0.5
    Q[3, 0, 1], Q[3, 1, 1] = float("inf"), float("nan")
    Q = Q.to(DEV)
    O = attend(c, Q, ot, 0.05, 2)
    assert bool(O[3].isnan().all())
    c.k[3], c.v[3] = c.k[3][:0], c.v[3][:0]
    O[3] = 0
    check(c, Q, O, 0.05, 2)


def test_infinite_feature_beside_a_padded_chunk():
    """Head dim 40: the second 32-wide chunk of features is padded; an infinite
    last feature must not meet the padding."""
    c = Cache([50], 1, 40, 16, 6)
    c.k[0] = c.k[0].abs()
    c.k[0][20, 0, 0] = float("-inf")
    c.write()
    Q = queries(1, 1, 40, BF16, 3).abs()
    O = attend(c, Q, F32, 0.3, 1)
    keep = [i for i in range(50) if i != 20]
    c.k[0], c.v[0] = c.k[0][keep], c.v[0][keep]
    check(c, Q, O, 0.3, 1)


def test_bad_pages_and_lengths_give_nan():
    """A page id outside the cache (negative, one behind the last, far out), a
    negative length and one beyond the table: NaN for that sequence, no access
    outside, and the other sequences untouched."""
    lens = [100, 100, 100, 100, 100, 100, 2000]
    c = Cache(lens, 2, 64, 16, 8, cap=2048 // 16).write()
    Q = queries(7, 4, 64, BF16, 8)
    good = attend(c, Q, BF16, 0.1, 4).clone()
    c.table[0, 3] = -1
    c.table[1, 6] = c.K.shape[0]
    c.table[2, 0] = (1 << 31) - 1
    c.table[6, 100] = -(1 << 31)
    lens2 = torch.tensor([100, 100, 100, -1, 2049, 100, 2000], dtype=torch.int32, device=DEV)
    O = attend(c, Q, BF16, 0.1, 4, lens=lens2)
    for b in range(7):
        if b == 5:
            assert torch.equal(O[b], good[b])
        else:
            assert bool(O[b].isnan().all()), b


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements, its last pages in use."""
    page, Hkv, D = 64, 2, 128
    n_pages = (1 << 31) // (page * Hkv * D) + 70000
    c = Cache([1000], Hkv, D, page, 11)
    used = c.K.shape[0]
    c.K = torch.empty(n_pages, Hkv, page, D, dtype=BF16, device=DEV)
    c.V = torch.empty(n_pages, Hkv, D, page, dtype=BF16, device=DEV)
    c.table = torch.where(c.table < used, c.table + (n_pages - used), c.table)
    c.write()
    Q = queries(1, 8, D, BF16, 2)
    check(c, Q, attend(c, Q, BF16, D ** -0.5, 8), D ** -0.5, 8)
    kv = torch.randn(1, 2 * Hkv * D, device=DEV)
    pos = torch.tensor([999], dtype=torch.int32, device=DEV)
    aa.aa_kv_append(kv[:, :Hkv * D], kv[:, Hkv * D:], c.K, c.V, c.table, pos)
    pg = int(c.table[0, 999 // page])
    assert torch.equal(c.K[pg, :, 999 % page], kv[0, :Hkv * D].view(Hkv, D).to(BF16))
    assert torch.equal(c.V[pg, :, :, 999 % page], kv[0, Hkv * D:].view(Hkv, D).to(BF16))


def test_more_than_65535_sequences():
    """Pages shared between sequences, as after a common prompt."""
    B, H, D, page, n_pages, scale = 70000, 2, 8, 16, 64, 0.5
    g = torch.Generator().manual_seed(6)
    K = torch.randn(n_pages, 1, page, D, generator=g).to(BF16).to(DEV)
    V = torch.randn(n_pages, 1, D, page, generator=g).to(BF16).to(DEV)
    table = torch.randint(0, n_pages, (B, 2), generator=g, dtype=torch.int32).to(DEV)
    lens = torch.randint(0, 2 * page + 1, (B,), generator=g, dtype=torch.int32).to(DEV)
    Q = queries(B, H, D, BF16, 3)
    O = torch.full((B, H, D), 77.0, device=DEV)
    aa.aa_attn_decode(Q, K, V, table, lens, O, scale)
    k = K[table.long(), 0].double().reshape(B, 1, 2 * page, D)
    v = V[table.long(), 0].double().transpose(2, 3).reshape(B, 1, 2 * page, D)
    qk = k * Q.view(B, H, 1, D).double()
    dead = (torch.arange(2 * page, device=DEV) >= lens[:, None])[:, None]
    s = (qk.sum(3) * scale).masked_fill(dead, -float("inf"))
    p = torch.softmax(s, 2).nan_to_num(0.0)
    ref = (p[..., None] * v).sum(2)
    # the bound of check(), of every sequence at once
    mag = (qk.abs().sum(3) * scale).masked_fill(dead, 0.0).amax(2)
    spread = s.amax(2) - s.masked_fill(dead, float("inf")).amin(2)
    eps_s = (3 * D + 3) * U * mag + 8 * U * (1 + spread.clamp_min(0.0))
    tol = (2 * eps_s + 2.0 ** -25 + 2 * (2 * page / 8 + 64) * U)[..., None] * (p[..., None] * v.abs()).sum(2)
    tol = tol + U * (ref.abs() + tol)
    assert bool(((O.double() - ref).abs() <= tol).all())


# ------------------------------------------------------------------- append ---

def test_append_of_a_long_prompt():
    """More values than the threads of one launch."""
    n, Hkv, D, page = 70000, 2, 128, 64
    pages = -(-n // page)
    g = torch.Generator().manual_seed(8)
    kv = torch.randn(n, 2 * Hkv * D, generator=g).to(BF16).to(DEV)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].to(DEV)
    K = torch.zeros(pages, Hkv, page, D, dtype=BF16, device=DEV)
    V = torch.zeros(pages, Hkv, D, page, dtype=BF16, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    aa.aa_kv_append(kv[:, :Hkv * D], kv[:, Hkv * D:], K, V, table, pos, torch.zeros_like(pos))
    gotK = K[table[0].long()].permute(0, 2, 1, 3).reshape(-1, Hkv * D)
    gotV = V[table[0].long()].permute(0, 3, 1, 2).reshape(-1, Hkv * D)
    assert torch.equal(gotK[:n], kv[:, :Hkv * D]) and torch.equal(gotV[:n], kv[:, Hkv * D:])
    assert not bool(gotK[n:].any()) and not bool(gotV[n:].any())


@pytest.mark.parametrize("Hkv,D,page,dt", [(32, 24, 64, F32), (1, 8, 16, BF16), (8, 128, 32, BF16), (3, 256, 16, F32)])
def test_append_prompts_then_tokens(Hkv, D, page, dt):
    """Whole prompts of several sequences in one call (rows of a wider QKV
    tensor), then one token each; padding and bad places are skipped, every
    other slot keeps its bits."""
    say("append", Hkv, D, page, dt)
    lens = [37, 1, 0, 64]
    c = Cache([n + 2 for n in lens], Hkv, D, page, 21, fill=3.0)
    g = torch.Generator().manual_seed(1)
    n, W = sum(lens) + 3, Hkv * D
    rows = torch.randn(n, W + 2 * W + 5, generator=g).to(dt).to(DEV)       # an odd row stride
    k, v = rows[:, W:2 * W], rows[:, 2 * W:3 * W]
    seq = [s for s, m in enumerate(lens) for _ in range(m)] + [0, 1 << 20, 3]
    pos = [j for m in lens for j in range(m)] + [-1, 0, c.most * page]      # padding, no such sequence, behind the table
    perm = torch.randperm(n, generator=g)
    seq, pos = (torch.tensor(t, dtype=torch.int32)[perm].to(DEV) for t in (seq, pos))
    wantK, wantV = c.K.clone(), c.V.clone()
    for t in range(n):
        s, p = int(seq[t]), int(pos[t])
        if 0 <= s < 4 and 0 <= p < c.most * page:
            pg = int(c.table[s, p // page])
            wantK[pg, :, p % page] = k[t].view(Hkv, D).to(BF16)
            wantV[pg, :, :, p % page] = v[t].view(Hkv, D).to(BF16)
    aa.aa_kv_append(k, v, c.K, c.V, c.table, pos, seq)
    torch.cuda.synchronize()
    assert torch.equal(c.K, wantK) and torch.equal(c.V, wantV)
    # one new token per sequence, sequence 1 sits this step out, sequence 2's page is not in the cache
    c.table[2, 0] = -5
    pos = torch.tensor([37, -1, 0, 64], dtype=torch.int32, device=DEV)
    for s in (0, 3):
        pg = int(c.table[s, int(pos[s]) // page])
        wantK[pg, :, int(pos[s]) % page] = k[s].view(Hkv, D).to(BF16)
        wantV[pg, :, :, int(pos[s]) % page] = v[s].view(Hkv, D).to(BF16)
    aa.aa_kv_append(rows[:4, W:2 * W].unflatten(1, (Hkv, D)), v[:4].unflatten(1, (Hkv, D)), c.K, c.V, c.table, pos)
    torch.cuda.synchronize()
    assert torch.equal(c.K, wantK) and torch.equal(c.V, wantV)


@pytest.mark.parametrize("Hkv,D,page,dt", [(3, 24, 16, F32), (2, 256, 128, BF16), (5, 8, 64, BF16), (1, 200, 32, F32)])
def test_append_at_once_equals_append_in_parts(Hkv, D, page, dt):
    """Prompts that begin at odd positions, padding, places outside the cache and
    tokens in no order: what a call writes does not depend on how many tokens it
    has, and nothing else changes."""
    say("append in parts", Hkv, D, page, dt)
    starts, lens = [5, 0, 1, 37, 64], [150, 200, 8, 97, 64]
    lens[0] += 8 * D                                                       # enough for the call that turns
    most = -(-max(s + n for s, n in zip(starts, lens)) // page)
    g = torch.Generator().manual_seed(D)
    pages = 5 * most + 3
    table = torch.randperm(pages, generator=g)[:5 * most].to(torch.int32).view(5, most)
    table[1, 1] = pages                                                    # no such page
    seq = [s for s, n in enumerate(lens) for _ in range(n)]
    pos = [b + j for b, n in zip(starts, lens) for j in range(n)]
    seq, pos = torch.tensor(seq, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32)
    pos[40:43] = -1
    pos[170] = most * page
    seq[175], seq[176] = 5, -1
    tail = torch.randperm(64, generator=g) + seq.numel() - 64              # the last prompt in no order
    seq[-64:], pos[-64:] = seq[tail], pos[tail]
    n, W = seq.numel(), Hkv * D
    rows = torch.randn(n, 2 * W + 3, generator=g).to(dt).to(DEV)
    k, v = rows[:, :W], rows[:, W:2 * W]
    table, seq, pos = table.to(DEV), seq.to(DEV), pos.to(DEV)
    K = [torch.full((pages, Hkv, page, D), 3.0, dtype=BF16, device=DEV) for _ in range(2)]
    V = [torch.full((pages, Hkv, D, page), 3.0, dtype=BF16, device=DEV) for _ in range(2)]
    aa.aa_kv_append(k, v, K[0], V[0], table, pos, seq)
    for lo in range(0, n, 31):
        aa.aa_kv_append(k[lo:lo + 31], v[lo:lo + 31], K[1], V[1], table, pos[lo:lo + 31], seq[lo:lo + 31])
    assert torch.equal(K[0], K[1]) and torch.equal(V[0], V[1])
    # and against plain indexing
    ok = (pos >= 0) & (pos < most * page) & (seq >= 0) & (seq < 5)
    t = ok.nonzero()[:, 0]
    pg = table[seq[t].long(), pos[t].long() // page].long()
    t, pg = t[pg < pages], pg[pg < pages]
    slot = pos[t].long() % page
    assert torch.equal(K[0][pg, :, slot], k[t].view(-1, Hkv, D).to(BF16))
    assert torch.equal(V[0][pg, :, :, slot], v[t].view(-1, Hkv, D).to(BF16))
    written = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    written[pg, slot] = True
    assert bool((K[0].transpose(1, 2)[~written] == 3).all()) and bool((V[0].permute(0, 3, 1, 2)[~written] == 3).all())


@pytest.mark.parametrize("n", [(1 << 30) - 64, (1 << 30) - 63, (1 << 30) - 1])
def test_append_of_the_most_tokens_of_a_grid(n):
    """Around 2^30 tokens, where the turned append's threads reach what a grid
    can count: the first tokens, one in the middle and the last are written, all
    others are padding."""
    say("append of many tokens", n)
    D, page = 8, 16
    rows = torch.zeros(n, D, dtype=BF16, device=DEV)            # keys and values alike
    pos = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    seq = torch.zeros(n, dtype=torch.int32, device=DEV)
    at = list(range(5)) + [n // 2 + 3, n - 2, n - 1]
    for j, t in enumerate(at):
        rows[t] = torch.arange(D, device=DEV) + 10 * (j + 1)
        pos[t] = j + 12                                         # over a page's end
    K = torch.full((4, 1, page, D), 3.0, dtype=BF16, device=DEV)
    V = torch.full((4, 1, D, page), 3.0, dtype=BF16, device=DEV)
    table = torch.tensor([[2, 1]], dtype=torch.int32, device=DEV)
    wantK, wantV = K.clone(), V.clone()
    for j, t in enumerate(at):
        pg, slot = (2, 1)[(j + 12) // page], (j + 12) % page
        wantK[pg, 0, slot] = rows[t]
        wantV[pg, 0, :, slot] = rows[t]
    aa.aa_kv_append(rows, rows, K, V, table, pos, seq)
    torch.cuda.synchronize()
    assert torch.equal(K, wantK) and torch.equal(V, wantV)


def test_append_then_attend_equals_a_written_cache():
    lens = [1, 33, 100]
    H, Hkv, D = 8, 2, 64
    c = Cache(lens, Hkv, D, 16, 31).write()
    Q = queries(3, H + 2 * Hkv, D, BF16, 4)
    want = attend(c, Q[:, :H * D], BF16, 0.125, H).clone()
    for b, n in enumerate(lens):      # take the last token out, append it again
        pg = int(c.table[b, (n - 1) // 16])
        c.K[pg, :, (n - 1) % 16] = float("nan")
        c.V[pg, :, :, (n - 1) % 16] = float("nan")
    k = torch.stack([t[-1] for t in c.k])
    v = torch.stack([t[-1] for t in c.v])
    aa.aa_kv_append(k, v, c.K, c.V, c.table, c.lens - 1)
    assert torch.equal(attend(c, Q[:, :H * D], BF16, 0.125, H), want)


def test_no_sequences_and_no_tokens():
    c = Cache([4], 1, 16, 16, 1)
    e = torch.empty(0, 16, device=DEV)
    none = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    z = torch.empty(0, dtype=torch.int32, device=DEV)
    aa.aa_kv_append(e, e, c.K, c.V, c.table, z)
    aa.aa_attn_decode(e, c.K, c.V, none, z, torch.empty(0, 1, 16, device=DEV), 1.0)


def test_graphs_streams_and_repeats():
    """An append and an attention captured together and replayed while lengths,
    positions and queries change in place; two graphs of other batches share one
    workspace; every replay equals the eager calls bit for bit."""
    H, Hkv, D, page = 8, 2, 64, 16
    caches = [Cache([900, 40], Hkv, D, page, 41, fill=0.0).write(), Cache([3000], Hkv, D, page, 42, fill=0.0).write()]
    ws = torch.empty(max(c.workspace(H).numel() for c in caches), dtype=torch.uint8, device=DEV)
    st = []
    for c in caches:
        B = len(c.k)
        st.append({"qkv": torch.randn(B, (H + 2 * Hkv) * D, device=DEV), "len": torch.full_like(c.lens, 17),
                   "pos": torch.full_like(c.lens, 16), "O": torch.zeros(B, H, D, device=DEV)})

    def step(c, s, O):
        q = s["qkv"]
        aa.aa_kv_append(q[:, H * D:(H + Hkv) * D], q[:, (H + Hkv) * D:], c.K, c.V, c.table, s["pos"])
        aa.aa_attn_decode(q[:, :H * D], c.K, c.V, c.table, s["len"], O, 0.125, ws)

    graphs = []
    for c, s in zip(caches, st):
        step(c, s, s["O"])
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(c, s, s["O"])
        graphs.append(gr)
    side = torch.cuda.Stream()
    for r in range(4):
        want = []
        for c, s in zip(caches, st):
            s["qkv"].normal_()
            s["len"].copy_(torch.clamp(c.lens - 3 * r, min=1))
            s["pos"].copy_(s["len"] - 1)
            O = torch.empty_like(s["O"])
            step(c, s, O)
            want.append(O)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for s, w in zip(st, want):
            assert torch.equal(s["O"], w), r
        O = torch.empty_like(st[0]["O"])
        with torch.cuda.stream(side):
            step(caches[0], st[0], O)
        side.synchronize()
        assert torch.equal(O, want[0])


def test_binding_refuses_before_the_library():
    c = Cache([20], 2, 32, 16, 1, fill=0.0)
    Q, O = torch.zeros(1, 4 * 32, device=DEV), torch.zeros(1, 4, 32, device=DEV)
    ws = c.workspace(4)
    with pytest.raises(ValueError, match="V|v_pages"):
        aa.aa_attn_decode(Q, c.K, c.K, c.table, c.lens, O, 1.0, ws)
    with pytest.raises(ValueError, match="shape"):
        aa.aa_attn_decode(Q[:, :64], c.K, c.V, c.table, c.lens, O, 1.0, ws)
    with pytest.raises(TypeError, match="dtype"):
        aa.aa_attn_decode(Q, c.K, c.V, c.table.long(), c.lens, O, 1.0, ws)
    with pytest.raises(ValueError, match="contiguous"):
        aa.aa_attn_decode(torch.zeros(1, 256, device=DEV)[:, ::2], c.K, c.V, c.table, c.lens, O, 1.0, ws)
    with pytest.raises(aa.AAError, match="divide"):
        aa.aa_attn_decode(torch.zeros(1, 3 * 32, device=DEV), c.K, c.V, c.table, c.lens, torch.zeros(1, 3, 32, device=DEV),
                          1.0, ws)
    with pytest.raises(aa.AAError, match="finite"):
        aa.aa_attn_decode(Q, c.K, c.V, c.table, c.lens, O, math.inf, ws)
    with pytest.raises(aa.AAError, match="page_size"):
        aa.aa_attn_decode(Q, c.K[:, :, :8].contiguous(), c.V[..., :8].contiguous(), c.table, c.lens, O, 1.0, ws)
    big = Cache([20000], 2, 32, 16, 1, fill=0.0)
    with pytest.raises(aa.AAError, match="workspace"):
        aa.aa_attn_decode(Q, big.K, big.V, big.table, big.lens, O, 1.0)
    with pytest.raises(aa.AAError, match="more tokens"):
        aa.aa_kv_append(torch.zeros(2, 64, device=DEV), torch.zeros(2, 64, device=DEV), c.K, c.V, c.table,
                        torch.zeros(2, dtype=torch.int32, device=DEV))
