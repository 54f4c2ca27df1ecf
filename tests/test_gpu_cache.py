"""Rotary positions, cache blocks and slots, appending in 8 bits and attention
over the 8-bit cache on the GPU, against the float64 oracle.

Bounds. u = 2^-24 is fp32's half step. Each is a worst-case count of roundings:
  rotary     the reduced angle is a fp32 number of half turns (off by at most
             u/2 of a half turn, so pi u/2 radians), sine and cosine within 2
             units (4 u), two products and a sum: |a| + |b| times 8 u, and the
             output's own half step for bf16 (2^-8)
  attention  with A = sum p |v|, N = sum |v| over the keys, S = max c sum |q| |k|
             and T = max c max |q| sum |k|:
             a score is off by at most (d + 8) 2 u S (sums in tensor cores
             keep at least 23 bits: 2 u a step), and shifts every weight by
             twice that; ex2 is off by 2^-22 for each weight, group and merge
             factor; sums over L keys run in steps of 16: (L / 16 + 64) 2 u A;
             the output's half step. Weights are rounded, the row's reference
             having weight 1, and small ones to the smallest number's half:
             fp32 queries, bf16 ones of more than 128 columns: two fp16 or one,
               2^-22 or 2^-11; scaled by at least 2^9 (2^13, less up to 2^4
               between blocks' scales), so 2^-25 / 2^9 = 2^-34 N;
             other bf16 queries, up to 16 rows per key/value head: fp16, then
               hi + lo / 16 in e4m3, 2^-11 and the 2^-4 of hi times that of lo,
               2^-8; scaled by at least 2^2 (2^7, less 2^4 between blocks'
               scales, less 2^1 as the reference may be above the largest
               weight), lo's smallest half is 2^-10 / 2^4, so 2^-16 N.
               Their query elements are hi + lo / 16 of a row whose largest is
               at least 2^7, exact but for lo's smallest half, 2^-14 of it,
               2^-21 T on a score
             more rows: fp16 weights, 2^-11, scaled by 2^7, 2^-25 / 2^7 N; values
               times their scale's ratio to a largest one, both rounded to fp16
               unless powers of two, 2^-11 each (the ratio is at least 2^-4 and
               an e4m3 number 2^-9: 2^-13 is not below fp16's normal numbers).
               Query elements are scaled to a largest of at least 2^14:
               2^-25 / 2^14 T
"""

import numpy as np
import pytest
import torch

from head_scaled_dot_gb300 import mha
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
OK, INVALID, FULL = 0, 1, 7


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mha.load()


def f64(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

ROTARY = [
    # B, T, h, h_kv, d, sections, interleaved, per_axis, inverse, farthest, dtype
    (2, 5, 4, 2, 128, [16, 24, 24], False, False, False, 1 << 20, "bf16"),
    (1, 1, 8, 8, 128, [64], False, False, False, (1 << 31) - 1, "bf16"),
    (3, 67, 3, 1, 64, [16, 16], True, True, True, 100, "f32"),
    (1, 33, 2, 2, 80, [7, 13], False, True, False, 5000, "f32"),     # 4-byte vectors, a rest
    (2, 9, 5, 5, 256, [10, 20, 30, 4], True, False, False, 1 << 24, "bf16"),
    (1, 200, 1, 1, 2, [1], True, False, False, 1000, "f32"),
    (2, 31, 2, 1, 6, [1, 2], False, False, True, 77, "bf16"),
    (1, 17, 40, 8, 96, [12, 12], False, True, False, 1 << 16, "bf16"),  # half of a row turns
    (4, 300, 12, 12, 64, [0, 32], False, False, False, 1 << 20, "f32"),
    (70, 3, 1, 1, 32, [3, 5, 8], True, True, False, 1 << 20, "f32"),
]


def rotary_inputs(case):
    B, T, h, h_kv, d, sections, _, _, _, far, dtype = case
    g = torch.Generator(device="cuda").manual_seed(d + T)
    Q = torch.randn((B, h, T, d), device="cuda", generator=g).to(DT[dtype])
    K = torch.randn((B, h_kv, T, d), device="cuda", generator=g).to(DT[dtype])
    pos = torch.randint(-far, far, (len(sections), B, T), device="cuda", generator=g).to(torch.int32)
    pos.view(-1)[-1] = far
    return Q, K, pos


def rotary_bound(X, ref, sections, interleaved, dtype):
    P = sum(sections)
    a = np.abs(f64(X))
    pair = a.copy()
    ia, ib = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else \
        (slice(0, P), slice(P, 2 * P))
    pair[..., ia] = pair[..., ib] = a[..., ia] + a[..., ib]
    tol = 8 * U * pair + (HALF_STEP["bf16"] * np.abs(ref) if dtype == "bf16" else 0)
    tol[..., 2 * P:] = 0  # columns that do not turn are copied
    return tol


@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "B%d_T%d_h%d_%d_d%d_%s" % (
    c[0], c[1], c[2], c[3], c[4], c[10]))
def test_rotary_matches_oracle(case):
    B, T, h, h_kv, d, sections, inter, per_axis, inverse, far, dtype = case
    Q, K, pos = rotary_inputs(case)
    steps = mha.rotary_steps(sections, per_axis=per_axis)
    f = co.rotary_frequencies(sections, 10000.0, per_axis)
    Qo, Ko = mha.rotary(Q, K, pos, steps, sections, inter, inverse)
    for X, Y in ((Q, Qo), (K, Ko)):
        ref = co.rotary(f64(X), pos.cpu().numpy(), f, sections, inter, inverse)
        # the oracle's own angle: position * frequency in float64
        own = far * 2.0 ** -53 * 2
        tol = rotary_bound(X, ref, sections, inter, dtype)
        assert (np.abs(f64(Y) - ref) <= tol * (1 + own / U)).all()
    # in place, and without K: the same bits
    Q2 = Q.clone()
    mha.rotary(Q2, None, pos, steps, sections, inter, inverse, out=(Q2, None))
    assert torch.equal(Q2, Qo)


def test_rotary_inverse_is_the_gradient():
    """g . rotary(x) is linear in x: its differences are exact up to rounding,
    and equal inverse(g)."""
    case = (1, 6, 2, 2, 16, [3, 5], False, True, False, 50, "f32")
    X, G, pos = rotary_inputs(case)
    steps = mha.rotary_steps([3, 5], per_axis=True)
    turn = lambda x, inv=False: mha.rotary(x, None, pos, steps, [3, 5], inverse=inv)[0]
    grad = f64(turn(G, True))
    g64 = f64(G)
    for e in range(0, X.numel(), 7):
        # x and x with element e set to 1 and 0: one output pair differs
        one, zero = X.clone(), X.clone()
        one.view(-1)[e], zero.view(-1)[e] = 1.0, 0.0
        diff = (g64 * (f64(turn(one)) - f64(turn(zero)))).sum()
        scale = np.abs(g64).max() * 2 * (1 + np.abs(f64(X)).max())
        assert abs(diff - grad.reshape(-1)[e]) <= 32 * U * scale
    back = turn(turn(X), True)
    assert (np.abs(f64(back - X)) <= 32 * U * np.abs(f64(X)).max()).all()


# ---------------------------------------------------------------------------
# Blocks and slots
# ---------------------------------------------------------------------------

def pool(cached, bt, n_blocks, max_blocks, seed):
    g = np.random.default_rng(seed)
    order = g.permutation(n_blocks)
    table = np.full((len(cached), max_blocks), -7)
    at = 0
    for b, L in enumerate(cached):
        k = -(-L // bt)
        table[b, :k] = order[at:at + k]
        at += k
    free = np.full(n_blocks, -9)
    free[:n_blocks - at] = order[at:]
    return table, free, n_blocks - at


RESERVE = [
    # B, most cached, n, bt, free blocks of what is needed, seed
    (1, 0, 1, 16, 2.0, 1), (5, 100, 40, 16, 1.0, 2), (64, 900, 1, 64, 1.0, 3),
    (33, 500, 300, 32, 0.5, 4), (1024, 60, 70, 48, 0.8, 5), (1024, 200, 1, 16, 0.3, 6),
    (7, 3000, 2000, 1, 1.0, 7), (300, 64, 9, 1024, 1.0, 8),
]


@pytest.mark.parametrize("case", RESERVE, ids=lambda c: "B%d_n%d_bt%d" % (c[0], c[2], c[3]))
def test_reserve_and_release_match_oracle(case):
    B, most, n, bt, share, seed = case
    g = np.random.default_rng(seed)
    cached = [int(x) for x in g.integers(0, most + 1, B)]
    new = [int(x) for x in g.integers(0, n + 1, B)]
    new[0] = n
    need = sum(-(-(a + m) // bt) - -(-a // bt) for a, m in zip(cached, new))
    held = sum(-(-a // bt) for a in cached)
    max_blocks = max(-(-(a + m) // bt) for a, m in zip(cached, new)) + 1
    n_blocks = held + max(1, int(need * share))
    table, free, n_free = pool(cached, bt, n_blocks, max_blocks, seed)
    want = co.reserve(cached, new, free, n_free, table, bt, n)
    tab, err = ints(table.tolist()), word()
    total, slots, left = mha.cache_reserve(ints(cached), ints(new), ints(free.tolist()),
                                           ints([n_free]), tab, bt, n, dev_error=err)
    assert total.tolist() == want[0]
    assert np.array_equal(slots.cpu().numpy(), want[1])
    assert left.tolist() == [want[2]]
    assert np.array_equal(tab.cpu().numpy(), want[3])
    assert mha.get_device_error(err) == (FULL if want[4] else OK)
    # every third sequence ends: its blocks come back on top of the stack
    done = [int(b % 3 == 0) for b in range(B)]
    stack = ints(free.tolist())
    total2, left2 = mha.cache_release(total, ints(done), stack, left, tab, bt, dev_error=err)
    ref_total, ref_free = co.release(want[0], done, free.tolist()[:want[2]], want[2], want[3], bt)
    assert total2.tolist() == ref_total and left2.tolist() == [len(ref_free)]
    assert stack.tolist()[:len(ref_free)] == ref_free
    assert mha.get_device_error(err) == OK


def test_reserve_refuses_bad_lengths_one_by_one():
    bt, n = 16, 8
    cached, new = [10, -1, 20, 0, 5, 60], [8, 2, 9, -3, 0, 8]
    table = np.full((6, 4), -1)
    table[0, 0], table[2, :2], table[4, 0], table[5] = 0, [1, 2], 3, [4, 5, 6, 7]
    free = list(range(8, 20))
    want = co.reserve(cached, new, free, 12, table, bt, n)
    assert want[5] and not want[4]
    tab, err = ints(table.tolist()), word()
    total, slots, left = mha.cache_reserve(ints(cached), ints(new), ints(free), ints([12]), tab,
                                           bt, n, dev_error=err)
    assert total.tolist() == want[0] == [18, -1, 20, 0, 5, 60]
    assert np.array_equal(slots.cpu().numpy(), want[1]) and left.tolist() == [11]
    assert mha.get_device_error(err) == INVALID
    # a count of free blocks outside the stack is held to it
    for n_free, kept in ((40, 11), (-3, 0)):
        _, slots, left = mha.cache_reserve(ints(cached), ints(new), ints(free), ints([n_free]),
                                           tab, bt, n, dev_error=err)
        assert left.tolist() == [kept] and mha.get_device_error(err) == INVALID
    # giving back more blocks than the pool has
    stack = ints(free)
    total, left = mha.cache_release(ints([64, 16]), ints([1, 1]), stack, ints([10]),
                                    ints([[0, 1, 2, 3], [4, 5, 6, 7]]), bt, dev_error=err)
    assert total.tolist() == [64, 16] and left.tolist() == [10] and stack.tolist() == free
    assert mha.get_device_error(err) == INVALID


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

class Cache:
    """A cache on the GPU with rows already in it, and the same in the oracle's form."""

    def __init__(self, n_blocks, h, bt, d_h, d_vh, seed, spread=4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bt = bt
        self.t, self.o = {}, {}
        for name, d in (("K", d_h), ("V", d_vh)):
            byte = torch.randint(0, 256, (n_blocks, h, bt, d), device="cuda", generator=g,
                                 dtype=torch.int64).to(torch.uint8)
            byte[(byte & 0x7f) == 0x7f] = 0x3a
            e = torch.randint(-spread, spread + 1, (n_blocks, h), device="cuda", generator=g)
            self.t[name] = byte
            self.t[name + "s"] = torch.exp2(e.float() - 5)
        self.sync()

    def sync(self):
        for name in ("K", "V"):
            self.o[name] = co.E4M3[self.t[name].cpu().numpy()]
            self.o[name + "s"] = f64(self.t[name + "s"])

    @property
    def args(self):
        return self.t["K"], self.t["V"], self.t["Ks"], self.t["Vs"]

    def append(self, K, V, slots, dev_error=None):
        mha.cache_append(K, V, slots, *self.args, dev_error=dev_error)
        for name, x in (("K", K), ("V", V)):
            co.append(f64(x), slots.cpu().numpy(), self.o[name], self.o[name + "s"], self.bt)

    def check(self):
        for name in ("K", "V"):
            got = co.E4M3[self.t[name].cpu().numpy()]
            assert np.array_equal(got, self.o[name], equal_nan=True), name
            assert np.array_equal(f64(self.t[name + "s"]), self.o[name + "s"]), name


def slots_of(cached, new, n, bt, n_blocks, seed):
    """Slots of ragged new rows, blocks scattered over the cache."""
    order = np.random.default_rng(seed).permutation(n_blocks)
    slots, at = np.full((len(cached), n), -1), 0
    for b, (L, a) in enumerate(zip(cached, new)):
        k = -(-(L % bt + a) // bt)
        p = L % bt + np.arange(a)
        slots[b, :a] = order[at + p // bt] * bt + p % bt
        at += k
    assert at <= n_blocks
    return torch.tensor(slots, dtype=torch.int64, device="cuda")


APPEND = [
    # cached, new, n, h, d_h, d_vh, bt, dtype
    ([0], [1], 1, 1, 16, 16, 16, "bf16"),
    ([5, 16, 31, 0], [1, 1, 1, 1], 1, 3, 128, 128, 16, "bf16"),
    ([3, 0, 63, 100], [200, 77, 1, 0], 200, 2, 128, 64, 64, "bf16"),
    ([0, 7, 15], [33, 40, 17], 40, 2, 80, 48, 16, "f32"),
    ([1000, 2], [30, 1100], 1100, 1, 256, 32, 1024, "f32"),
    ([90], [500], 501, 1, 96, 256, 48, "bf16"),
    ([17] * 40, [3] * 40, 3, 4, 64, 64, 32, "f32"),
    ([1], [300], 300, 2, 256, 256, 256, "bf16"),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "B%d_n%d_d%d_%d_bt%d_%s" % (
    len(c[0]), c[2], c[4], c[5], c[6], c[7]))
def test_append_matches_oracle(case):
    cached, new, n, h, d_h, d_vh, bt, dtype = case
    g = torch.Generator(device="cuda").manual_seed(n + d_h)
    n_blocks = sum(-(-(L % bt + a) // bt) for L, a in zip(cached, new)) + 3
    cache = Cache(n_blocks, h, bt, d_h, d_vh, n)
    K = torch.randn((len(cached), h, n, d_h), device="cuda", generator=g)
    # values of widely different sizes: scales rise, and small ones go subnormal
    V = torch.randn((len(cached), h, n, d_vh), device="cuda", generator=g)
    V *= torch.exp2(torch.randint(-12, 6, V.shape[:3], device="cuda", generator=g).float())[..., None]
    err = word()
    cache.append(K.to(DT[dtype]), V.to(DT[dtype]), slots_of(cached, new, n, bt, n_blocks, n), err)
    cache.check()
    assert mha.get_device_error(err) == OK


def test_append_infinities_nan_zeros_and_denormals():
    h, d, bt = 2, 16, 16
    cache = Cache(4, h, bt, d, d, 3)
    K = torch.zeros((1, h, 20, d), device="cuda")
    K[0, 0, 3, 5], K[0, 0, 4, 1], K[0, 0, 5, 2], K[0, 0, 6] = np.inf, -np.inf, np.nan, 3.0
    K[0, 1, 17] = 1e-42           # fp32 denormals, in the second block
    V = torch.full((1, h, 20, d), 3e38, device="cuda")
    V[0, 1] = 448.0 * 2.0 ** 40
    V[0, 1, 0, 0] = 450.0 * 2.0 ** 40   # just past a power of two's range
    slots = slots_of([0], [20], 20, bt, 4, 1)
    cache.append(K, V, slots)
    cache.check()
    a = int(slots[0, 3]) // bt
    assert cache.o["K"][a, 0, 3, 5] == 448 and cache.o["K"][a, 0, 4, 1] == -448
    assert np.isnan(cache.o["K"][a, 0, 5, 2]) and cache.o["Ks"][a, 0] == 2.0 ** -7
    # more rows into the second block: its kept rows are rounded to the new scale
    more = torch.arange(4, 10, device="cuda")[None] + slots[0, 16]
    cache.append(torch.randn((1, h, 6, d), device="cuda"), torch.randn((1, h, 6, d), device="cuda"),
                 more)
    cache.check()


def test_append_row_by_row_equals_append_at_once():
    h, d, bt, n = 2, 32, 32, 40
    g = torch.Generator(device="cuda").manual_seed(9)
    # all above 2^-6 of the largest scale: no value is rounded twice to another one
    K = torch.randn((1, h, n, d), device="cuda", generator=g).sign() * (
        1 + torch.rand((1, h, n, d), device="cuda", generator=g))
    K *= torch.exp2(torch.arange(n, device="cuda") % 7.0)[None, None, :, None]
    slots = slots_of([0], [n], n, bt, 2, 2)
    once, rows = Cache(2, h, bt, d, d, 1), Cache(2, h, bt, d, d, 1)
    once.append(K, K, slots)
    for i in range(n):
        rows.append(K[:, :, i:i + 1].contiguous(), K[:, :, i:i + 1].contiguous(),
                    slots[:, i:i + 1].contiguous())
    once.check()
    rows.check()
    at = torch.arange(n, device="cuda")
    for name in ("K", "V"):
        x, y = (f64(c.t[name].view(torch.float8_e4m3fn)) * f64(c.t[name + "s"])[:, :, None, None]
                for c in (once, rows))
        for s in slots[0].tolist():
            assert np.array_equal(x[s // bt, :, s % bt], y[s // bt, :, s % bt])


def test_append_leaves_rows_without_a_proper_slot_unwritten():
    h, d, bt = 1, 16, 16
    cache = Cache(4, h, bt, d, d, 4)
    before = {k: v.clone() for k, v in cache.t.items()}
    x = torch.randn((5, h, 4, d), device="cuda")
    slots = torch.tensor([[-1, 5, 6, 7],          # no first row: nothing
                          [64, 65, 66, 67],       # past the cache
                          [1 << 40, -1, -1, -1],  # far past it
                          [16, 17, 40, 18],       # the third row does not follow
                          [-1, -1, -1, -1]], device="cuda")
    err = word()
    mha.cache_append(x, x, slots, *cache.args, dev_error=err)
    assert mha.get_device_error(err) == INVALID
    good = torch.tensor([[16, 17, -1, -1]], device="cuda")
    ref = Cache(4, h, bt, d, d, 4)
    ref.append(x[3:4].contiguous(), x[3:4].contiguous(), good)
    for name in ("K", "V"):
        got, want = cache.t[name], before[name]
        for blk in (0, 2, 3):
            assert torch.equal(got[blk], want[blk])
        assert torch.equal(got[1, :, 2], want[1, :, 2]) and torch.equal(got[1, :, 4:], want[1, :, 4:])
        assert torch.equal(got[1, :, :2], ref.t[name][1, :, :2])


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def table_of(total, bt, n_blocks, max_blocks, seed, fill=-1):
    order = np.random.default_rng(seed).permutation(n_blocks)
    table, at = np.full((len(total), max_blocks), fill), 0
    for b, L in enumerate(total):
        k = -(-max(0, L) // bt)
        table[b, :k] = order[at:at + k]
        at += k
    return table


def attention_bound(ref, parts, d, longest, dtype, rows=1):
    """d: the larger head size; rows: query rows per key/value head."""
    A, S, N, T = parts
    score = (d + 8) * 2 * U * S
    if dtype == "bf16" and d <= 128:
        if rows <= 16:
            weight, floor, q = 2.0 ** -8 + 2.0 ** -11, 2.0 ** -16, 2.0 ** -21
        else:
            weight, floor, q = 3 * 2.0 ** -11, 2.0 ** -32, 2.0 ** -39
        score = score + T * q
    else:
        weight, floor = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22, 2.0 ** -34
    return (HALF_STEP[dtype] * np.abs(ref) + floor * N
            + A * (weight + 2 * 2 * score + 4 * 2.0 ** -22 + (longest / 16 + 64) * 2 * U))


def attend_and_check(cache, total, new, n_q, h, d_h, d_vh, dtype, tail, seed, table=None, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, bt, n_blocks = len(total), cache.bt, cache.t["K"].shape[0]
    Q = torch.randn((B, h, n_q, d_h), device="cuda", generator=g).to(DT[dtype])
    if table is None:
        table = table_of(total, bt, n_blocks, max(1, max(-(-t // bt) for t in total)), seed)
    c = d_h ** -0.5
    err = word()
    Z = mha.attention_cache(Q, *cache.args, ints(table.tolist()), ints(total), c,
                            new_len=None if new is None else ints(new), causal_tail=tail,
                            dev_error=err, **kw)
    assert mha.get_device_error(err) == OK
    ref, parts = co.attention_cache(f64(Q), cache.o["K"], cache.o["V"], cache.o["Ks"],
                                   cache.o["Vs"], table, total, new or [n_q] * B, c, tail)
    tol = attention_bound(ref, parts, max(d_h, d_vh), max(total), dtype, n_q * h // cache.t["K"].shape[1])
    got = f64(Z)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    # rows that see nothing are exact zeros
    assert (got[parts[2] == 0] == 0).all()
    return Q, Z


ATTEND = [
    # total, new, n_q, h, h_kv, d_h, d_vh, bt, dtype, tail
    ([1], None, 1, 1, 1, 16, 16, 16, "bf16", True),
    ([300, 17, 16, 1], None, 1, 4, 4, 128, 128, 16, "bf16", True),
    ([2000], None, 1, 2, 2, 64, 64, 64, "bf16", False),
    ([700, 65], [3, 1], 3, 8, 2, 128, 128, 32, "bf16", True),
    ([333, 5, 0, 90], [5, 5, 5, 0], 5, 4, 1, 96, 80, 48, "bf16", True),
    ([40, 9], [9, 9], 9, 8, 2, 64, 128, 16, "bf16", True),         # three tiles of rows
    ([500, 31], None, 2, 2, 2, 256, 256, 32, "bf16", True),
    ([500, 31], None, 16, 4, 4, 256, 48, 16, "bf16", True),
    ([1025, 64], None, 2, 3, 3, 64, 64, 16, "f32", True),
    ([129, 700], [7, 2], 7, 4, 2, 128, 112, 64, "f32", True),
    ([77], None, 12, 2, 2, 32, 256, 1024, "f32", False),
    ([20, 3], [20, 5], 20, 2, 1, 64, 64, 16, "bf16", True),        # all rows new; more than total
    ([3000], [150], 150, 2, 1, 64, 64, 128, "bf16", True),
    ([100] * 70, None, 1, 2, 1, 32, 32, 16, "bf16", True),
    ([12000, 700], [17, 20], 20, 4, 4, 128, 128, 64, "bf16", True),  # some groups of keys per CTA
    ([5000, 700], [70, 64], 70, 16, 4, 128, 112, 32, "bf16", True),
    ([900, 2500], [64, 1], 64, 2, 1, 64, 48, 16, "bf16", True),      # one tile of rows exactly
    ([900, 2500], None, 129, 1, 1, 80, 128, 16, "bf16", False),      # one row past it
    ([600, 0, 130, 2000], [600, 0, 400, 257], 600, 3, 1, 64, 64, 16, "bf16", True),  # heads across tiles
    ([1500, 1], [1400, 1], 1400, 2, 2, 32, 32, 32, "bf16", True),    # most tiles see few keys
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "B%d_L%d_nq%d_h%d_%d_d%d_%d_bt%d_%s" % (
    len(c[0]), c[0][0], c[2], c[3], c[4], c[5], c[6], c[7], c[8]))
def test_attention_matches_oracle(case):
    total, new, n_q, h, h_kv, d_h, d_vh, bt, dtype, tail = case
    n_blocks = sum(-(-t // bt) for t in total) + 2
    cache = Cache(n_blocks, h_kv, bt, d_h, d_vh, total[0])
    attend_and_check(cache, total, new, n_q, h, d_h, d_vh, dtype, tail, total[0])


def test_attention_of_the_largest_batch_and_of_none():
    total = [b % 40 for b in range(1024)]
    cache = Cache(3 * 1024, 1, 16, 32, 32, 11)
    attend_and_check(cache, total, None, 1, 2, 32, 32, "bf16", True, 12)
    attend_and_check(cache, [0] * 5, None, 2, 2, 32, 32, "bf16", True, 13)
    attend_and_check(cache, total, None, 9, 2, 32, 32, "bf16", True, 14)
    attend_and_check(cache, [0] * 5, None, 200, 1, 32, 32, "bf16", True, 15)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_with_scales_of_every_size(dtype):
    """Blocks whose values differ by 2^60: the smallest weights meet the
    largest values."""
    cache = Cache(30, 2, 16, 64, 64, 21, spread=0)
    e = torch.arange(30, device="cuda").float()[:, None] % 7
    cache.t["Vs"].copy_(torch.exp2(e * 10 - 30).expand(30, 2))
    cache.t["Ks"].copy_(torch.exp2(-e - 4).expand(30, 2))
    cache.sync()
    attend_and_check(cache, [450, 3], None, 2, 2, 64, 64, dtype, True, 22)


@pytest.mark.parametrize("n_q", [2, 20, 150])
def test_attention_of_many_keys_with_scales_of_every_size(n_q):
    """As above with many groups of keys, and with zero and negative scales."""
    cache = Cache(200, 2, 16, 64, 64, 23, spread=0)
    e = torch.arange(200, device="cuda").float()[:, None] % 7
    cache.t["Vs"].copy_(torch.exp2(e * 10 - 30).expand(200, 2))
    cache.t["Ks"].copy_(torch.exp2(-e - 4).expand(200, 2))
    cache.sync()
    attend_and_check(cache, [2900, 150], None, n_q, 2, 64, 64, "bf16", True, 24)
    cache.t["Vs"][::5] = 0
    cache.t["Ks"][1::5] *= -1
    cache.t["Ks"][2::5] = 0
    cache.sync()
    attend_and_check(cache, [2900, 150], None, n_q, 2, 64, 64, "bf16", True, 24)


@pytest.mark.parametrize("n_q", [20, 150])
def test_nan_and_stale_rows_with_many_rows(n_q):
    bt, d, h = 16, 64, 2
    total = [n_q + 203]
    cache = Cache(30, h, bt, d, d, 33)
    table = table_of(total, bt, 30, 24, 5, fill=1 << 30)
    at = lambda p: (int(table[0, p // bt]), slice(None), p % bt)
    for p in range(total[0], -(-total[0] // bt) * bt):  # past the end
        cache.t["K"][at(p)] = 0x7f
        cache.t["V"][at(p)] = 0xff
    cache.sync()
    Q, clean = attend_and_check(cache, total, None, n_q, h, d, d, "bf16", True, 34, table)
    args = (ints(table.tolist()), ints(total), d ** -0.5)
    # rows are positions 203 on: row 9 is the first that sees the value, 12 the key
    cache.t["V"][at(212)][..., 5] = 0xff
    Z = mha.attention_cache(Q, *cache.args, *args, causal_tail=True)
    assert torch.equal(Z[:, :9], clean[:, :9])
    nan = torch.isnan(Z[:, 9:]).reshape(1, n_q - 9, h, d)
    assert nan[..., 5].all() and not nan[..., :5].any() and not nan[..., 6:].any()
    cache.t["K"][at(215)] = 0x7f
    Z = mha.attention_cache(Q, *cache.args, *args, causal_tail=True)
    assert torch.equal(Z[:, :9], clean[:, :9])
    assert torch.isnan(Z[:, 12:]).all() and not torch.isnan(Z[:, 9:12, :5]).any()


def test_stale_rows_and_nan_do_not_reach_rows_that_do_not_see_them():
    bt, d, h = 16, 64, 2
    cache = Cache(8, h, bt, d, d, 31)
    total, n_q = [50], 6
    table = table_of(total, bt, 8, 6, 5, fill=1 << 30)  # entries past the end: nowhere
    at = lambda p: (int(table[0, p // bt]), slice(None), p % bt)
    # rows past the end hold NaN; so do key row 47 and value row 48
    for p in range(50, 64):
        cache.t["K"][at(p)] = 0x7f
        cache.t["V"][at(p)] = 0xff
    cache.sync()
    Q, clean = attend_and_check(cache, total, None, n_q, h, d, d, "bf16", True, 32, table)
    cache.t["K"][at(47)] = 0x7f
    cache.t["V"][at(48)][..., 5] = 0xff
    Z = mha.attention_cache(Q, *cache.args, ints(table.tolist()), ints(total), d ** -0.5,
                            causal_tail=True)
    # rows are positions 44 .. 49: the first three see neither
    assert torch.equal(Z[:, :3], clean[:, :3])
    assert torch.isnan(Z[:, 3:]).all()
    cache.t["K"][at(47)] = 0x20
    cache.sync()
    _, fine = attend_and_check_nan_free(cache, total, n_q, h, d, table, Q)
    got = fine.view(1, n_q, h, d)
    assert torch.isnan(got[:, 4:, :, 5]).all()
    keep = [x for x in range(d) if x != 5]
    assert torch.isfinite(got[:, 4:][..., keep]).all() and torch.isfinite(got[:, :4]).all()


def attend_and_check_nan_free(cache, total, n_q, h, d, table, Q):
    return Q, mha.attention_cache(Q, *cache.args, ints(table.tolist()), ints(total), d ** -0.5,
                                  causal_tail=True)


def test_attention_reads_no_block_outside_the_cache():
    """Blocks out of range are left out and recorded, lengths are held to the table."""
    bt, d, h = 16, 64, 2
    cache = Cache(6, h, bt, d, d, 41)
    Q = torch.randn((2, h, 1, d), device="cuda").bfloat16()
    table = [[0, 1, 2], [3, 99, 4]]
    err = word()
    Z = mha.attention_cache(Q, *cache.args, ints(table), ints([48, 40]), 0.125, dev_error=err)
    assert mha.get_device_error(err) == INVALID
    # the second sequence without its bad block: 16 + 8 keys
    ref, parts = co.attention_cache(f64(Q[1:]), cache.o["K"], cache.o["V"], cache.o["Ks"],
                                   cache.o["Vs"], np.array([[3, 4]]), [24], [1], 0.125, False)
    assert (np.abs(f64(Z[1:]) - ref) <= attention_bound(ref, parts, d, 24, "bf16")).all()
    for bad in ([1000, 40], [48, -5]):
        Z = mha.attention_cache(Q, *cache.args, ints([[0, 1, 2], [3, 5, 4]]), ints(bad), 0.125,
                                dev_error=err)
        assert mha.get_device_error(err) == INVALID and torch.isfinite(Z.float()).all()
    full = mha.attention_cache(Q, *cache.args, ints([[0, 1, 2], [3, 5, 4]]), ints([48, 0]), 0.125)
    assert torch.equal(Z, full)


def test_attention_is_the_same_whatever_the_workspace_holds():
    cache = Cache(70, 2, 32, 128, 128, 51)
    total, n_q, h = [900, 1200], 2, 4
    table = ints(table_of(total, 32, 70, 40, 6).tolist())
    Q = torch.randn((2, h, n_q, 128), device="cuda").bfloat16()
    ws = torch.full((mha.attention_cache_workspace_size(2, n_q, h, 2, 128, 128),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (0xFF, 0x00, 0x7F):
        ws.fill_(fill)
        outs.append(mha.attention_cache(Q, *cache.args, table, ints(total), 0.1, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("n_q,share", [(1, 1), (4, 4), (200, 4), (20, 4)])
def test_calls_in_a_row_end_and_agree(n_q, share):
    """Many groups per CTA, call after call without a wait between them: no
    wait inside the kernel runs out, and every call gives the same bits."""
    B, h_kv, L, bt = 2, 4, 6000, 64
    cache = Cache(2 * -(-L // bt) + 1, h_kv, bt, 128, 128, 91)
    table = ints(table_of([L, L - 77], bt, 2 * -(-L // bt) + 1, -(-L // bt), 8).tolist())
    Q = torch.randn((B, h_kv * share, n_q, 128), device="cuda").bfloat16()
    lens, err = ints([L, L - 77]), word()
    out = [mha.attention_cache(Q, *cache.args, table, lens, 0.09, causal_tail=True, dev_error=err)
           for _ in range(40)]
    assert mha.get_device_error(err) == OK
    assert all(torch.equal(z, out[0]) for z in out)


def test_offsets_past_32_bits():
    """A cache of more than 4 GB of keys: rows written to and read from its end."""
    n_blocks, h, bt, d_h, d_vh = 36000, 8, 64, 256, 16
    K = torch.empty((n_blocks, h, bt, d_h), dtype=torch.uint8, device="cuda")
    V = torch.empty((n_blocks, h, bt, d_vh), dtype=torch.uint8, device="cuda")
    Ks, Vs = (torch.empty((n_blocks, h), device="cuda") for _ in range(2))
    assert K.numel() > 1 << 32
    n = 100
    g = torch.Generator(device="cuda").manual_seed(61)
    kx = torch.randn((1, h, n, d_h), device="cuda", generator=g).bfloat16()
    vx = torch.randn((1, h, n, d_vh), device="cuda", generator=g).bfloat16()
    table = [[n_blocks - 1, n_blocks - 3]]
    pos = np.arange(n)
    slots = torch.tensor(np.array(table[0])[pos // bt] * bt + pos % bt, device="cuda")[None]
    mha.cache_append(kx, vx, slots.contiguous(), K, V, Ks, Vs)
    Q = torch.randn((1, h, 1, d_h), device="cuda", generator=g).bfloat16()
    Z = mha.attention_cache(Q, K, V, Ks, Vs, ints(table), ints([n]), 0.0625)
    small = [co.E4M3[x[table[0]].cpu().numpy()] for x in (K, V)]
    sc = [f64(x[table[0]]) for x in (Ks, Vs)]
    oc = [np.zeros_like(x) for x in small], [np.zeros_like(x) for x in sc]
    at = (pos // bt * bt + pos % bt)[None]
    for i, x in enumerate((kx, vx)):
        co.append(f64(x), at, oc[0][i], oc[1][i], bt)
        flat = lambda y: y.transpose(1, 0, 2, 3).reshape(h, 2 * bt, -1)[:, :n]
        assert np.array_equal(flat(small[i]), flat(oc[0][i])) and np.array_equal(sc[i], oc[1][i])
    ref, parts = co.attention_cache(f64(Q), small[0], small[1], sc[0], sc[1], np.array([[0, 1]]), [n], [1],
                                   0.0625, False)
    assert (np.abs(f64(Z) - ref) <= attention_bound(ref, parts, d_h, n, "bf16")).all()


@pytest.mark.parametrize("n_q", [2, 40, 150])
def test_calls_on_another_stream_and_two_graphs_that_share_a_workspace(n_q):
    cache = Cache(40, 2, 32, 64, 64, 71)
    total, h = [600, 500], 2
    table = ints(table_of(total, 32, 40, 20, 7).tolist())
    lens = ints(total)
    Q = [torch.randn((2, h, n_q, 64), device="cuda").bfloat16() for _ in range(2)]
    want = [mha.attention_cache(q, *cache.args, table, lens, 0.125, causal_tail=True) for q in Q]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mha.attention_cache(Q[0], *cache.args, table, lens, 0.125, causal_tail=True, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    ws = torch.empty(mha.attention_cache_workspace_size(2, n_q, h, 2, 64, 64), dtype=torch.uint8,
                     device="cuda")
    outs, graphs = [torch.empty_like(w) for w in want], []
    for q, o in zip(Q, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mha.attention_cache(q, *cache.args, table, lens, 0.125, causal_tail=True, out=o,
                                workspace=ws)
        graphs.append(g)
    for k in (0, 1, 1, 0, 1):
        outs[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k], want[k])
    # the lengths are read when a graph is replayed
    lens.copy_(ints([33, 1]))
    graphs[0].replay()
    torch.cuda.synchronize()
    now = mha.attention_cache(Q[0], *cache.args, table, lens, 0.125, causal_tail=True)
    assert torch.equal(outs[0], now) and not torch.equal(now, want[0])


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own, few and many rows, many times over."""
    cache = Cache(80, 2, 64, 128, 128, 73)
    total, h = [2400, 2300], 4
    table, lens = ints(table_of(total, 64, 80, 38, 9).tolist()), ints(total)
    Q = [torch.randn((2, h, n, 128), device="cuda").bfloat16() for n in (1, 8, 40, 200)]
    want = [mha.attention_cache(q, *cache.args, table, lens, 0.09, causal_tail=True) for q in Q]
    torch.cuda.synchronize()
    err, streams, got = word(), [torch.cuda.Stream() for _ in Q], [[] for _ in Q]
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(mha.attention_cache(Q[k], *cache.args, table, lens, 0.09,
                                                  causal_tail=True, dev_error=err))
    torch.cuda.synchronize()
    assert mha.get_device_error(err) == OK
    assert all(torch.equal(z, want[k]) for k in range(len(Q)) for z in got[k])


# ---------------------------------------------------------------------------
# A run of them together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_prompt_and_generation_steps_through_the_whole_chain(graph):
    """Projection, rotary, reserve, append, attention, output projection: a
    ragged prompt and then single tokens, every stage against the oracle on the
    library's own inputs of that stage. With `graph` the step is captured once
    and replayed while the sequences grow."""
    B, h, d, dm, bt, n_blocks, max_blocks = 3, 4, 64, 128, 16, 24, 6
    sections, c = [8, 12, 12], 0.125
    g = torch.Generator(device="cuda").manual_seed(81)
    W = [torch.randn((dm, h * d), device="cuda", generator=g).bfloat16() / 11 for _ in range(3)]
    W_O = (torch.randn((h * d, dm), device="cuda", generator=g) / 16).bfloat16()
    steps = mha.rotary_steps(sections)
    cache = Cache(n_blocks, h, bt, d, d, 82)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
    free, n_free = torch.arange(n_blocks, dtype=torch.int32, device="cuda"), ints([n_blocks])
    cached, err = ints([0] * B), word()
    # the oracle's own blocks
    o = dict(table=np.full((B, max_blocks), -1), n_free=n_blocks, cached=[0] * B)

    def stages(X, new, pos, n):
        Q, K, V = mha.qkv_projection(X, None, *W, h, d, d)
        Qr, Kr = mha.rotary(Q, K, pos, steps, sections)
        total, slots, left = mha.cache_reserve(cached, new, free, n_free, table, bt, n,
                                               dev_error=err)
        mha.cache_append(Kr, V, slots, *cache.args, dev_error=err)
        Z = mha.attention_cache(Qr, *cache.args, table, total, c, new_len=new, causal_tail=True,
                                dev_error=err)
        Y = mha.output_projection(Z, W_O, h, d)
        cached.copy_(total)
        n_free.copy_(left)
        return Q, K, V, Qr, Kr, total, slots, Z, Y

    def check(out, X, new, pos, n):
        Q, K, V, Qr, Kr, total, slots, Z, Y = out
        f = co.rotary_frequencies(sections)
        for a, b in ((Q, Qr), (K, Kr)):
            ref = co.rotary(f64(a), pos.cpu().numpy(), f, sections)
            assert (np.abs(f64(b) - ref) <= rotary_bound(a, ref, sections, False, "bf16")).all()
        want = co.reserve(o["cached"], new, free.tolist(), o["n_free"], o["table"], bt, n)
        o["cached"], o["n_free"], o["table"] = want[0], want[2], want[3]
        assert total.tolist() == want[0] and np.array_equal(slots.cpu().numpy(), want[1])
        assert np.array_equal(table.cpu().numpy(), want[3])
        for name, x in (("K", Kr), ("V", V)):
            co.append(f64(x), want[1], cache.o[name], cache.o[name + "s"], bt)
        cache.check()
        ref, parts = co.attention_cache(f64(Qr), cache.o["K"], cache.o["V"], cache.o["Ks"],
                                       cache.o["Vs"], want[3], want[0], new, c, True)
        assert (np.abs(f64(Z) - ref) <= attention_bound(ref, parts, d, max(want[0]), "bf16", n)).all()
        y = f64(Z) @ f64(W_O)
        size = np.abs(f64(Z)) @ np.abs(f64(W_O))
        assert (np.abs(f64(Y) - y) <= HALF_STEP["bf16"] * np.abs(y) + 512 * U * size).all()
        assert mha.get_device_error(err) == OK

    T, new = 40, [40, 17, 1]
    X = torch.randn((B, T, dm), device="cuda", generator=g).bfloat16()
    pos = torch.arange(T, device="cuda", dtype=torch.int32).expand(3, B, T).contiguous()
    check(stages(X, ints(new), pos, T), X, new, pos, T)

    X1 = torch.randn((B, 1, dm), device="cuda", generator=g).bfloat16()
    one, pos1 = ints([1] * B), torch.zeros((3, B, 1), dtype=torch.int32, device="cuda")
    run = lambda: stages(X1, one, pos1, 1)
    if graph:
        recorded = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(recorded):
            out = run()
    for step in range(20):
        X1.copy_(torch.randn((B, 1, dm), device="cuda", generator=g))
        pos1.copy_(cached[None, :, None].expand(3, B, 1))
        if graph:
            recorded.replay()
        else:
            out = run()
        torch.cuda.synchronize()
        check(out, X1, [1] * B, pos1, 1)
    # a finished sequence's blocks come back
    held = -(-o["cached"][0] // bt)
    total, left = mha.cache_release(cached, ints([1, 0, 0]), free, n_free, table, bt, dev_error=err)
    assert total.tolist() == [0] + o["cached"][1:] and left.tolist() == [o["n_free"] + held]
    assert mha.get_device_error(err) == OK
