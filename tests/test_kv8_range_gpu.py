"""The 8-bit cache's attention where its arithmetic runs out of range: factors that underflow,
one key that holds most of a long context's softmax, query rows with an outlier channel.

The bounds count roundings, of sizes relative to what is rounded, so that none grows into the
result itself: output in bf16 (2^-8 of it); each probability in fp16 (2^-11 of it), which ends
25 bits below 1, with the row's largest probability times value scale at 2^12 or above (2^-37 of
that), in the kernel of groups of more than 128 rows at 2^7 or above (2^-32); 2^-23 of the accumulator for every 16 keys that the tensor cores add to it; the
exponential's 2^-20; and the error of the scores, twice (in the probability and in the sum)."""
import math

import numpy as np
import pytest
import torch

from tests import kv8_reference as ref
from tests import test_kv8_gpu as base
from tests.test_kv8_gpu import DEV, ints, kv8  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def reference(q, pool, scales, pages, last, scale, group):
    """64-bit attention on the GPU of the rows q [n][hq][D] of one sequence, row t over the keys
    0 .. last[t] of its pages: out, lse and the bounds of their errors.  group: rows per kv head of the call."""
    n, hq, D = q.shape
    hkv = pool.shape[1]
    values, idx = torch.from_numpy(ref.VALUES).to(DEV), torch.from_numpy(ref.key_index(D)).to(DEV)
    L = int(max(last)) + 1
    pages = torch.as_tensor(pages, device=DEV).long()[:-(-L // 16)]
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=DEV)
    tol_lse = torch.zeros((n, hq), dtype=torch.float64, device=DEV)
    sees = torch.arange(L, device=DEV)[None] <= torch.as_tensor(last, device=DEV)[:, None]
    for h in range(hkv):
        x = values[pool[pages, h].long()] * scales[pages, h].double()[..., None]
        k = x[:, 0][:, idx].reshape(-1, D)[:L]
        v = x[:, 1].view(-1, D, 16).transpose(1, 2).reshape(-1, D)[:L]
        sv = scales[pages, h, 1].double().repeat_interleave(16)[:L]
        for i in range(h * hq // hkv, (h + 1) * hq // hkv):
            a = q[:, i].double()
            s = (a @ k.T * scale).masked_fill(~sees, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.where(sees, torch.exp(s - torch.where(top.isinf(), 0.0, top)), 0.0)
            l = p.sum(-1, keepdim=True)
            some = l > 0
            lse[:, i] = torch.where(some, top + torch.log(l), -math.inf)[:, 0]
            out[:, i] = torch.where(some, p @ v / l, 0.0)
            # scores: fp32 products and sums; queries as two terms, which are exact down to 2^-13 of the
            # row's largest element and off by 2^-21 of it below
            small = (a.abs() < 2.0 ** -13 * a.abs().amax(-1, keepdim=True)) & (a != 0)
            ds = abs(scale) * (2.0 ** -21 * a.abs().amax(-1, keepdim=True) * (small.double() @ k.abs().T)
                               + 2.0 ** -23 * D * (a.abs() @ k.abs().T))
            ds = torch.where(sees, ds + 2.0 ** -22 * (1 + s.abs().nan_to_num(posinf=0)), 0.0).amax(-1, keepdim=True)
            mass = p @ v.abs() / l
            tol[:, i] = torch.where(some, 2.0 ** -8 * out[:, i].abs() + mass * (2.0 ** -11 + 2.0 ** -20 + L * 2.0 ** -27 + 2 * ds)
                                    + 2.0 ** (-37 if group <= 128 else -32) * (p * sv).amax(-1, keepdim=True) * (v.abs() / sv[:, None]).sum(0) / l, 0.0)
            # the sum: one fp32 addition a key
            tol_lse[:, i] = (2 * ds + 2.0 ** -20 + L * 2.0 ** -24)[:, 0] + 2.0 ** -22 * lse[:, i].abs().nan_to_num(posinf=0)
    return out, lse, tol, tol_lse


def check(out, lse, q, pool, scales, pages, last, scale=None, n=None):
    """n: tokens of the sequence, where q is not all of them."""
    D = q.shape[2]
    want, wl, tol, tol_lse = reference(q, pool, scales, pages, last, 1 / D ** 0.5 if scale is None else scale,
                                           (n or q.shape[0]) * q.shape[1] // pool.shape[1])
    assert not torch.isnan(out).any()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (float((err - tol).max()), float((err.norm(dim=-1) / want.norm(dim=-1)).nan_to_num().max()))
    inf = torch.isinf(wl)
    assert torch.equal(torch.isneginf(lse), inf)
    el = torch.where(inf, 0.0, lse.double() - torch.where(inf, 0.0, wl)).abs()
    assert (el <= tol_lse).all(), float((el - tol_lse).max())


# ---- factors below the smallest float -------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 5, 140])
@pytest.mark.parametrize("L", [1, 17, 130, 333])
@pytest.mark.parametrize("zero", ["q", "k", "both"])
def test_zero_queries_and_keys_give_the_mean(kv8, zero, L, n, D):  # noqa: F811
    """All scores are zero: the mean of the values that a row sees, whatever scale the append
    gave a page without a key above zero; rows that see nothing are zeros."""
    g = torch.Generator(device=DEV).manual_seed(L + n)
    hq, hkv, pages = 8, 2, -(-L // 16)
    pool, scales = kv8.new_cache(pages, hkv, D)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    k = torch.randn(L, hkv, D, generator=g, device=DEV).bfloat16() * (zero == "q")
    v = (1 + torch.randn(L, hkv, D, generator=g, device=DEV)).bfloat16()
    q = torch.randn(n, hq, D, generator=g, device=DEV).bfloat16() * (zero == "k")
    kv8.append(pool, scales, table, ints([0, L]), ints([L]), k, v)
    lse = torch.empty(n, hq, device=DEV)
    out = kv8.attention(q, pool, scales, table, ints([0, n]), ints([L]), lse=lse)
    check(out, lse, q, pool, scales, range(pages), [L - n + t for t in range(n)])


@pytest.mark.parametrize("n", [3, 140])
@pytest.mark.parametrize("size", [1.0, 1e-3, 2.0 ** -60])
def test_scale_zero_with_small_numbers(kv8, size, n):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(n)
    hq, hkv, D, L = 8, 2, 128, 333
    pool, scales = kv8.new_cache(21, hkv, D)
    table = torch.arange(21, dtype=torch.int32, device=DEV).view(1, -1)
    k, v = (torch.randn(L, hkv, D, generator=g, device=DEV) for _ in range(2))
    q = (torch.randn(n, hq, D, generator=g, device=DEV) * size).bfloat16()
    kv8.append(pool, scales, table, ints([0, L]), ints([L]), k * size, v)
    for scale in (0.0, -0.0, 1e-30):
        lse = torch.empty(n, hq, device=DEV)
        out = kv8.attention(q, pool, scales, table, ints([0, n]), ints([L]), scale=scale, lse=lse)
        check(out, lse, q, pool, scales, range(21), [L - n + t for t in range(n)], scale)


# ---- a key that holds most of the softmax ---------------------------------------------------

def sink_cache(g, L, hkv, D, at, sink_value):
    """One context of L keys that all sequences read: keys near zero but the one at `at`, which
    is 1 along every dimension; values 1 + noise, that key's `sink_value`."""
    pages = -(-L // 16)
    k = torch.randn(L, 1, hkv * D, generator=g, device=DEV).view(L, hkv, D) * 2.0 ** -8
    v = 1 + 0.25 * torch.randn(L, hkv, D, generator=g, device=DEV)
    k[at], v[at] = 1.0, sink_value
    return pages, k, v


@pytest.mark.parametrize("L,D", [(2048, 128), (8192, 64), (16384, 128), (32768, 64), (32760, 128), (131072, 128)])
@pytest.mark.parametrize("n", [1, 9, 32, 40])          # 4, 36 and 128 rows per kv head, and a prompt chunk
def test_one_key_with_most_of_the_softmax(kv8, L, D, n):  # noqa: F811
    """An attention sink before a long flat context.  19 sequences of 8 kv heads are as many groups as
    there are runs, so that each run holds a group from end to end."""
    g = torch.Generator(device=DEV).manual_seed(L + n)
    B, hkv, G = 19, 8, 4
    for at, sink_value in ((0, 0.0), (L // 2, 1.0)):
        pages, k, v = sink_cache(g, L, hkv, D, at, sink_value)
        pool, scales = kv8.new_cache(pages, hkv, D)
        table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
        kv8.append(pool, scales, table, ints([0, L]), ints([L]), k, v)
        for share in (0.5, 0.9, 0.99):
            # q . k / sqrt(D) of the sink against the others' zero: its share of the sum
            gap = math.log(share / (1 - share) * (L - 1))
            q = (torch.full((B * n, hkv * G, D), gap / D ** 0.5, device=DEV)
                 + 0.02 * torch.randn(B * n, hkv * G, D, generator=g, device=DEV)).bfloat16()
            lse = torch.empty(B * n, hkv * G, device=DEV)
            out = kv8.attention(q, pool, scales, table.expand(B, pages).contiguous(), ints(np.arange(B + 1) * n), ints([L] * B), lse=lse)
            for b in (0, 7):
                for t in sorted({0, n - 1}):
                    r = slice(b * n + t, b * n + t + 1)
                    check(out[r], lse[r], q[r], pool, scales, range(pages), [L - n + t], n=n)


@pytest.mark.parametrize("n", [1, 9, 32, 200])
def test_one_key_with_most_of_the_softmax_split(kv8, n):  # noqa: F811
    """The same for one sequence, whose groups are split over many runs and joined."""
    g = torch.Generator(device=DEV).manual_seed(n)
    hkv, G, L, D = 2, 4, 30000, 128
    pages, k, v = sink_cache(g, L, hkv, D, 5, 0.0)
    pool, scales = kv8.new_cache(pages, hkv, D)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    kv8.append(pool, scales, table, ints([0, L]), ints([L]), k, v)
    for share in (0.5, 0.9, 0.99):
        gap = math.log(share / (1 - share) * (L - 1))
        q = torch.full((n, hkv * G, D), gap / D ** 0.5, device=DEV).bfloat16()
        lse = torch.empty(n, hkv * G, device=DEV)
        out = kv8.attention(q, pool, scales, table, ints([0, n]), ints([L]), lse=lse)
        check(out[-1:], lse[-1:], q[-1:], pool, scales, range(pages), [L - 1], n=n)


@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (5, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("seqs", list(base.ATT))
def test_attention_without_a_floor(kv8, seqs, hq, hkv, D):  # noqa: F811
    """Ordinary and sharp softmaxes over pages of scales octaves apart, to the same bound."""
    rng = np.random.default_rng(len(seqs) + hq + D)
    for amp, spread in ((1.5, 2), (20.0, 2), (1.0, 9)):
        rs, kv, table, pool, scales = base.make_cache(rng, base.ATT[seqs], hkv, D, True, spread)
        q = torch.from_numpy(rng.standard_normal((int(rs[-1]), hq, D)) * amp).to(torch.bfloat16).to(DEV)
        pd, sd = torch.from_numpy(pool).to(DEV), torch.from_numpy(scales).to(DEV)
        lse = torch.empty(q.shape[:2], device=DEV)
        out = kv8.attention(q, pd, sd, ints(table), ints(rs), ints(kv), lse=lse)
        for b, (n, L) in enumerate(base.ATT[seqs]):
            r = slice(int(rs[b]), int(rs[b + 1]))
            if n and L:
                check(out[r], lse[r], q[r], pd, sd, table[b], [L - n + t for t in range(n)])
            else:
                assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()


# ---- query rows with an outlier -------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [3, 140])
@pytest.mark.parametrize("size", [100.0, 4096.0])
def test_queries_with_an_outlier_channel(kv8, size, n, D):  # noqa: F811
    """One channel of the queries is far larger than the others and the keys are zero there: the
    others decide the scores."""
    rng = np.random.default_rng(n + D)
    hq, hkv, L = 8, 2, 500
    rs, kv, table, pool, scales = base.make_cache(rng, [(n, L)], hkv, D)
    pool[:, :, 0][:, :, ref.key_index(D)[:, 3]] = 0
    q = rng.standard_normal((n, hq, D)) * 2
    q[:, :, 3] = size * np.sign(q[:, :, 3])
    q = torch.from_numpy(q).to(torch.bfloat16).to(DEV)
    pd, sd = torch.from_numpy(pool).to(DEV), torch.from_numpy(scales).to(DEV)
    lse = torch.empty(q.shape[:2], device=DEV)
    out = kv8.attention(q, pd, sd, ints(table), ints(rs), ints(kv), lse=lse)
    check(out, lse, q, pd, sd, table[0], [L - n + t for t in range(n)])


# ---- the same bits every time ---------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 9, 32, 40])
def test_repeated_calls_give_the_same_bits(kv8, n, D):  # noqa: F811
    """Whole groups of 16 tiles, 300 calls: a tile whose slots are used again too early would show as
    other values of a few dimensions."""
    g = torch.Generator(device=DEV).manual_seed(n + D)
    B, hkv, G, L = 19, 8, 4, 2048
    pages, k, v = sink_cache(g, L, hkv, D, 0, 0.0)
    pool, scales = kv8.new_cache(pages, hkv, D)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    kv8.append(pool, scales, table, ints([0, L]), ints([L]), k, v)
    q = torch.randn(B * n, hkv * G, D, generator=g, device=DEV).bfloat16()
    args = (q, pool, scales, table.expand(B, pages).contiguous(), ints(np.arange(B + 1) * n), ints([L] * B))
    first, again = kv8.attention(*args), torch.empty_like(q)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(300):
        kv8.attention(*args, out=again)
        wrong += (again != first).any()
    assert int(wrong) == 0
