"""The 8-bit cache with a scale per (block, kv head): append, block copy and decode
against the fp64 definition.  Codes and scales are compared bit for bit; attention
within the bound that step_ops.attention_bound derives."""
import ctypes as C

import numpy as np
import pytest

from oracle import step_ops
from test_abi import _gpu_visible

CODES = ["e4m3", "int8"]


def torch_mod():
    import torch
    return torch


def code_dtype(code):
    torch = torch_mod()
    return torch.float8_e4m3fn if code == "e4m3" else torch.int8


def to_pool(values, code):
    """Code values (float64, exact) as a device tensor of codes."""
    torch = torch_mod()
    t = torch.from_numpy(np.ascontiguousarray(values)).cuda()
    return t.to(torch.int8) if code == "int8" else t.float().to(torch.float8_e4m3fn)


def to_values(pool):
    return pool.float().cpu().numpy().astype(np.float64)


def bf16(x):
    torch = torch_mod()
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def same(got, want):
    """Equal numbers, NaN for NaN (e4m3 -0 and 0 count as equal)."""
    return np.array_equal(got, want, equal_nan=True)


def random_pool(rng, nb, H, d, code, spread=1.0):
    """Pools as appends leave them: values of every block rounded under its scale."""
    x = rng.standard_normal((nb, H, 16, d)) * np.exp(spread * rng.standard_normal((nb, H, 1, 1)))
    scales = np.vectorize(lambda a: step_ops.need_scale(a, code))(np.abs(x).max((2, 3))) if nb else np.zeros((0, H))
    return step_ops.round_code(x / scales[:, :, None, None], code), scales.astype(np.float32)


# ------------------------------------------------------------------------ refusals (no GPU)
@pytest.mark.skipif(_gpu_visible(), reason="passes placeholder device addresses: only where no GPU is reachable")
def test_host_validation(pa):
    L, p, odd = pa._lib, C.c_void_p(0x10000), C.c_void_p(0x10008)
    D = lambda nb=8, hkv=2, bs=16, d=128, dt=pa.PA_INT8: C.byref(pa.CacheDesc(nb, hkv, bs, d, dt, 1.0, 1.0))
    w = lambda k=p, ks=256, vs=256, T=1, kc=p, sc=p, slots=p, desc=None: L.pa_cache_write_scaled(
        k, p, ks, vs, slots, T, kc, p, sc, p, desc or D(), None, None)
    bad, uns = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    for kw in (dict(k=None), dict(k=odd), dict(ks=255), dict(vs=252), dict(ks=260), dict(T=-1), dict(kc=None), dict(kc=odd),
               dict(sc=None), dict(sc=C.c_void_p(0x10002)), dict(slots=None), dict(desc=D(hkv=0)), dict(desc=D(nb=-1))):
        assert w(**kw) == bad, kw
    for kw in (dict(bs=32), dict(d=96), dict(dt=pa.PA_BF16), dict(dt=pa.PA_F32), dict(dt=9)):
        assert w(desc=D(**kw)) == uns, kw
    assert w(T=0) == pa.PA_OK
    assert L.pa_copy_blocks_scaled(p, p, p, p, None, 1, D(), None, None) == bad
    assert L.pa_copy_blocks_scaled(p, p, p, p, p, -1, D(), None, None) == bad
    assert L.pa_copy_blocks_scaled(p, p, p, p, None, 0, D(), None, None) == pa.PA_OK
    need = pa.pa_decode_scaled_workspace_size(8, 2, 128)
    dec = lambda q=p, S=4, hq=8, mb=8, ctx=100, ws=p, wsb=need, desc=None, out=p: L.pa_decode_scaled(
        q, p, p, p, p, p, mb, p, ctx, S, hq, 0.1, ws, wsb, out, desc or D(), None, None)
    for kw in (dict(q=None), dict(q=odd), dict(S=-1), dict(hq=3), dict(hq=0), dict(mb=-1), dict(ctx=-1), dict(ctx=129),
               dict(ws=None), dict(ws=odd), dict(wsb=need - 1), dict(out=odd)):
        assert dec(**kw) == bad, kw
    assert dec(hq=32) == uns and dec(S=16385) == uns and dec(desc=D(dt=pa.PA_BF16)) == uns
    assert dec(S=16384, mb=1 << 27, ctx=(1 << 31) - 1) == uns
    assert dec(S=0) == pa.PA_OK
    assert pa.pa_decode_scaled_workspace_size(3, 2, 128) == 0


def test_binding_refuses_wrong_tensors(pa):
    torch = torch_mod()
    pool, sc = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        pa.pa_cache_write_scaled(x, x, slots, pool.float(), pool.float(), sc, sc)
    for k, s, scales in ((x.float(), slots, sc), (x, slots.int(), sc), (x, slots, sc.double()), (x, slots, sc[:, :1]),
                         (x[:, :1], slots, sc), (x.transpose(1, 2).contiguous().transpose(1, 2), slots, sc),
                         (x, slots, sc)):                       # the last: right, but not on a GPU
        with pytest.raises(AssertionError):
            pa.pa_cache_write_scaled(k, k, s, pool, pool, scales, sc)


# ------------------------------------------------------------------------ append
def run_write(pa, k, v, slots, kp, vp, ks, vs, code):
    """k, v: bf16 device tensors.  Returns the pools' values, scales and the flag."""
    torch = torch_mod()
    gk, gv = to_pool(kp, code), to_pool(vp, code)
    gks, gvs = torch.from_numpy(ks.copy()).cuda(), torch.from_numpy(vs.copy()).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_cache_write_scaled(k, v, torch.from_numpy(slots).cuda(), gk, gv, gks, gvs, err)
    flag = pa.pa_wait(err)
    return [to_values(gk), to_values(gv), gks.cpu().numpy(), gvs.cpu().numpy()], flag


def check_write(pa, k, v, slots, kp, vp, ks, vs, code):
    got, flag = run_write(pa, k.cuda(), v.cuda(), slots, kp, vp, ks, vs, code)
    want = [kp.copy(), vp.copy(), ks.copy(), vs.copy()]
    for x, i in ((k, 0), (v, 1)):
        step_ops.cache_write_scaled(x.double().numpy(), slots, want[i], want[2 + i], code)
    for g, w, what in zip(got, want, ("keys", "values", "key scales", "value scales")):
        assert same(g, w), what
    return got, flag


def appended(rng, nb, lens, counts):
    """Slots of counts[s] tokens behind lens[s], each sequence in blocks of its own."""
    ids = rng.permutation(nb)
    slots, at = [], 0
    for n, c in zip(lens, counts):
        first, last = n // 16, -(-(n + c) // 16)
        own = ids[at:at + last - first]
        at += last - first
        slots += [int(own[t // 16 - first]) * 16 + t % 16 for t in range(n, n + c)]
    assert at <= nb
    return np.array(slots, np.int64)


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("H,d", [(1, 64), (2, 128), (3, 64), (8, 128)])
@pytest.mark.parametrize("counts", [(1,), (1, 1, 1, 1, 1), (16,), (17, 1, 5), (40, 3, 100, 1, 0, 16)])
def test_append_matches_the_definition(pa, code, H, d, counts):
    rng = np.random.default_rng(H * 100 + d + len(counts))
    lens = rng.integers(0, 40, len(counts))
    nb = sum(-(-int(n + c) // 16) - int(n) // 16 for n, c in zip(lens, counts)) + 2
    kp, ks = random_pool(rng, nb, H, d, code)
    vp, vs = random_pool(rng, nb, H, d, code)
    slots = appended(rng, nb, lens.tolist(), counts)
    T = len(slots)
    # tokens far larger and far smaller than what the blocks hold: scales grow, or stay
    x = lambda: bf16(rng.standard_normal((T, H, d)) * np.exp(2.5 * rng.standard_normal((T, 1, 1))))
    got, flag = check_write(pa, x(), x(), slots, kp, vp, ks, vs, code)
    assert flag == 0


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_append_many_tokens_per_warp(pa, code):
    """Over the size at which a warp looks after 16 tokens: padding, tokens of a block in
    descending and mixed order, blocks that end anywhere in a window."""
    rng = np.random.default_rng(3)
    H, d, nb = 8, 64, 400
    counts = [1] * 40 + [16, 33, 700, 1, 5, 900, 450] + [1] * 20
    lens = rng.integers(0, 16, len(counts)).tolist()
    slots = appended(rng, nb, lens, counts)
    runs = np.split(slots, np.nonzero(np.diff(slots // 16))[0] + 1)
    out = []
    for i, r in enumerate(runs):
        out += [r[::-1] if i % 3 == 0 else rng.permutation(r)]
        if i % 5 == 0:
            out += [np.full(i % 4, -1)]
    slots = np.concatenate(out).astype(np.int64)
    assert len(slots) * H * 2 > 32768
    kp, ks = random_pool(rng, nb, H, d, code)
    x = lambda: bf16(rng.standard_normal((len(slots), H, d)) * np.exp(rng.standard_normal((len(slots), 1, 1))))
    _, flag = check_write(pa, x(), x(), slots, kp, kp, ks, ks, code)
    assert flag == 0


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("H,d", [(2, 128), (8, 64)])
@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("order", ["ascending", "twice"])
def test_append_runs_of_a_block(pa, code, H, d, big, order):
    """Runs in ascending order (of every length and first slot), and runs that name slots up to
    three times (with the same row each time, so that it does not matter which one lands), in
    calls where a warp looks after one token and after 16."""
    rng = np.random.default_rng(17)
    nb = 16000 // H if big else 140
    runs = []
    for b in rng.permutation(nb):
        first = int(rng.integers(0, 16))
        run = b * 16 + np.arange(first, int(rng.integers(first + 1, 17)))
        runs.append(run if order == "ascending" else rng.permutation(np.repeat(run, rng.integers(1, 4, len(run)))))
    slots = np.concatenate(runs).astype(np.int64)
    assert (len(slots) * H * 2 > 32768) == big
    kp, ks = random_pool(rng, nb, H, d, code)
    rows = rng.standard_normal((nb * 16, H, d)) * np.exp(2 * rng.standard_normal((nb * 16, 1, 1)))
    _, flag = check_write(pa, bf16(rows[slots]), bf16(-rows[slots]), slots, kp, kp, ks, ks, code)
    assert flag == 0


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_append_edge_values(pa, code):
    """Zeros, infinities, NaN, subnormal and huge numbers, exact ties and exact maxima,
    stored scales that are no scale, padding and slots outside the pool."""
    rng = np.random.default_rng(8)
    H, d, nb = 2, 64, 24
    rows = np.zeros((14, H, d), np.float32)
    rows[1] = np.inf
    rows[2, :, ::2] = np.nan
    rows[2, :, 1::2] = 3.0
    rows[3, :, :5] = [np.inf, -np.inf, np.nan, 1e-3, -2.0]
    rows[4] = 1e-40                                    # subnormal: below the smallest scale
    rows[5] = 2.0 ** -64 * 100
    rows[6] = 3e38
    rows[7] = step_ops.TOP[code] * 2.0 ** 5            # the largest code exactly
    rows[8] = step_ops.TOP[code] * 2.0 ** 5 * (1 + 2.0 ** -7)
    grid = np.unique(step_ops.round_code(np.linspace(-step_ops.TOP[code], step_ops.TOP[code], 4001), code))
    ties = (grid[:-1] + grid[1:]) / 2
    rows[9] = rng.choice(ties, (H, d))
    rows[9, :, 0] = step_ops.TOP[code]
    rows[10:] = rng.standard_normal((4, H, d))
    slots = np.array([16 * i for i in range(10)] + [16 * 12 + 3, 16 * 13 + 3, 16 * 14 + 3, 16 * 15 + 3], np.int64)
    kp, ks = random_pool(rng, nb, H, d, code)
    ks[12], ks[13], ks[14], ks[15] = np.nan, 0.0, np.inf, -1.0
    for s, flagged in ((slots, 0), (np.where(np.arange(14) % 3 == 1, -1, slots), 0),
                       (np.where(np.arange(14) == 5, nb * 16, slots), pa.PA_DEVERR_SLOT),
                       (np.where(np.arange(14) == 5, 2 ** 62, slots), pa.PA_DEVERR_SLOT)):
        _, flag = check_write(pa, bf16(rows), bf16(rows[::-1].copy()), s.astype(np.int64), kp, kp, ks, ks, code)
        assert flag == flagged


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_append_of_views_and_again(pa, code):
    """Keys and values as views of one fused projection; the same call again changes
    nothing; a slot named twice holds one of its tokens."""
    torch = torch_mod()
    rng = np.random.default_rng(4)
    H, d, nb = 4, 128, 9
    kp, ks = random_pool(rng, nb, H, d, code)
    slots = appended(rng, nb, [5, 30, 2], (20, 1, 40))
    fused = bf16(rng.standard_normal((len(slots), 3 * H, d)) * 4).cuda()
    q, k, v = fused.split([H, H, H], 1)
    first, _ = run_write(pa, k, v, slots, kp, kp, ks, ks, code)
    want, _ = check_write(pa, k.cpu(), v.cpu(), slots, kp, kp, ks, ks, code)
    assert all(same(a, b) for a, b in zip(first, want))
    again, _ = run_write(pa, k, v, slots, *first, code)
    assert all(same(a, b) for a, b in zip(first, again))
    x = bf16(rng.standard_normal((40, H, d))).cuda()
    twice = np.full(40, 16 * 3 + 7, np.int64)
    got, flag = run_write(pa, x, x, twice, kp, kp, ks, ks, code)
    assert flag == 0
    sigma = got[2][3]
    at = [i for i in range(40) if same(got[0][3, :, 7], step_ops.round_code(x[i].double().cpu().numpy() / sigma[:, None], code))]
    assert at


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("H,d", [(1, 64), (8, 128)])
def test_copy_blocks(pa, code, H, d):
    torch = torch_mod()
    rng = np.random.default_rng(2)
    kp, ks = random_pool(rng, 12, H, d, code)
    vp, vs = random_pool(rng, 12, H, d, code)
    pairs = np.array([[0, 5], [0, 6], [11, 1], [12, 2], [3, -1]], np.int32)
    t = [to_pool(kp, code), to_pool(vp, code), torch.from_numpy(ks.copy()).cuda(), torch.from_numpy(vs.copy()).cuda()]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_copy_blocks_scaled(*t, torch.from_numpy(pairs).cuda(), err)
    assert pa.pa_wait(err) == pa.PA_DEVERR_PAIR
    for got, a in zip(t, (kp, vp, ks, vs)):
        want = a.copy()
        for s, dst in pairs[:3]:
            want[dst] = a[s]
        assert same(got.float().cpu().numpy().astype(np.float64), want.astype(np.float64))


# ------------------------------------------------------------------------ decode
class Decode:
    def __init__(self, pa, code, hq, hkv, d, lens, seed=0, spread=1.0, extra_rows=0):
        torch = torch_mod()
        rng = np.random.default_rng(seed)
        self.pa, self.code, self.lens = pa, code, np.asarray(lens, np.int32)
        S = len(lens)
        self.blocks = [max(0, -(-int(n) // 16)) for n in lens]
        nb = sum(self.blocks) + 3
        self.kp, self.ks = random_pool(rng, nb, hkv, d, code, spread)
        self.vp, self.vs = random_pool(rng, nb, hkv, d, code, spread)
        ids = rng.permutation(nb)
        self.mb = max(1, max(self.blocks, default=1)) + 1
        self.tables = np.full((S, self.mb), -1, np.int32)
        at = 0
        for s, n in enumerate(self.blocks):
            self.tables[s, :n] = ids[at:at + n]
            at += n
            if lens[s] % 16:            # what stands behind the last token must not matter
                b = self.tables[s, n - 1]
                junk = np.nan if code == "e4m3" else -127.0
                self.kp[b, :, lens[s] % 16:] = junk
                self.vp[b, :, lens[s] % 16:] = junk
        for b in ids[at:]:              # blocks of nobody
            self.ks[b] = self.vs[b] = np.nan
        self.q = bf16(rng.standard_normal((S, hq, d)) * 1.5)
        self.scale = d ** -0.5
        self.out = torch.full((S + extra_rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((pa.pa_decode_scaled_workspace_size(hq, hkv, d),), 0xFF, dtype=torch.uint8, device="cuda")
        c = lambda a: torch.from_numpy(a).cuda()
        self.t = [to_pool(self.kp, code), to_pool(self.vp, code), c(self.ks), c(self.vs), c(self.tables), c(self.lens)]
        self.qd = self.q.cuda()

    def call(self, **kw):
        S = len(self.lens)
        a = dict(tables=self.t[4], lens=self.t[5], max_context=self.mb * 16, out=self.out[:S]) | kw
        self.pa.pa_decode_scaled(self.qd, *self.t[:4], a["tables"], a["lens"], a["max_context"], self.scale, a["out"],
                                 self.ws, self.err, a.get("stream"))

    def check(self, rows=None):
        S = len(self.lens)
        rows = np.arange(S) if rows is None else rows
        ref, mass, reach = step_ops.decode_scaled(self.q.double().numpy()[rows], self.kp, self.vp, self.ks, self.vs,
                                                  self.tables[rows], self.lens[rows], self.scale)
        got = self.out[:S].double().cpu().numpy()[rows]
        vmax = float(np.nan_to_num(np.abs(self.vp) * self.vs[:, :, None, None]).max(initial=0.0))
        far = np.abs(got - ref) - step_ops.attention_bound(ref, mass, reach, (int(self.lens.max(initial=0)), 2.0 ** -11, vmax))
        assert np.isfinite(got).all() and (far <= 0).all(), f"off by {far.max():.3g} more than the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (2, 1, 128), (8, 2, 128), (8, 1, 64), (16, 2, 128), (6, 3, 64), (5, 5, 128)])
@pytest.mark.parametrize("lens", [(1,), (0,), (16,), (0, 1, 15, 16, 17, 33, 100, 0, 512, 511), (2500, 3), tuple(range(0, 80, 3))])
def test_decode_matches_the_definition(pa, code, hq, hkv, d, lens):
    t = Decode(pa, code, hq, hkv, d, lens, seed=hq + d + len(lens), extra_rows=2)
    t.call()
    assert pa.pa_wait(t.err) == 0
    t.check()
    assert (t.out[len(lens):] == 7).all()      # rows behind the last sequence


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_decode_blocks_of_very_different_size(pa, code):
    """Scales far apart within a sequence, for keys and for values."""
    rng = np.random.default_rng(1)
    for d in (64, 128):
        t = Decode(pa, code, 8, 2, d, [400, 37, 1200], seed=9, spread=0.5)
        live = ~np.isnan(t.ks)
        for s, lo, hi in ((t.vs, -40, 40), (t.ks, -30, 2)):
            s[live] *= 2.0 ** rng.integers(lo, hi, live.sum())
        torch = torch_mod()
        t.t[2], t.t[3] = torch.from_numpy(t.ks).cuda(), torch.from_numpy(t.vs).cuda()
        # the bound's last term takes the largest value of the pool: per sequence here
        t.call()
        assert pa.pa_wait(t.err) == 0
        ref, mass, reach = step_ops.decode_scaled(t.q.double().numpy(), t.kp, t.vp, t.ks, t.vs, t.tables, t.lens, t.scale)
        got = t.out.double().cpu().numpy()
        assert np.isfinite(got).all()
        # f16 weights below 2^-14 of the reference lose 2^-25 of it, and the reference is
        # the largest p * sigma_v so far: 2^-25 * sum_t of the largest p sigma_v * |code| <= n 2^-25 * 448 * max(mass)
        far = np.abs(got - ref) - step_ops.attention_bound(ref, mass, reach, (0, 2.0 ** -11, 0.0))
        far -= np.array([[[n * 2.0 ** -25 * 512]] for n in t.lens]) * mass.max(2, keepdims=True) * 16
        assert (far <= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_decode_large_and_small_queries(pa, code):
    """Queries far outside f16's range (a zero one among them), a scale that undoes them."""
    torch = torch_mod()
    for power in (40, -40):
        t = Decode(pa, code, 4, 2, 128, [100, 7, 64], seed=5)
        t.q = (t.q.float() * 2.0 ** power).to(torch.bfloat16)
        t.q[1, 2] = 0
        t.qd, t.scale = t.q.cuda(), t.scale * 2.0 ** -power
        t.call()
        assert pa.pa_wait(t.err) == 0
        t.check()


@pytest.mark.gpu
def test_decode_many_sequences(pa):
    """More sequences than prefix sums in shared memory."""
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 40, 9001)
    t = Decode(pa, "int8", 2, 1, 64, lens, seed=6)
    t.call()
    assert pa.pa_wait(t.err) == 0
    t.check(np.concatenate([np.arange(50), rng.integers(0, 9001, 200), np.arange(8950, 9001)]))


@pytest.mark.gpu
def test_decode_many_blocks_per_warp(pa):
    """Over 32 blocks of a segment in one warp, and segments that span CTAs."""
    t = Decode(pa, "e4m3", 4, 4, 64, [40000] * 6 + [5, 12345, 0, 777], seed=7)
    t.call()
    assert pa.pa_wait(t.err) == 0
    t.check()


@pytest.mark.gpu
def test_decode_offsets_beyond_32_bits(pa):
    """A pool of more than 2^31 bytes whose blocks in use lie at its end."""
    torch = torch_mod()
    hkv, d, nb = 8, 128, 150_000
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kc = torch.zeros(nb, hkv, 16, d, dtype=torch.int8, device="cuda")
    vc = torch.zeros(nb, hkv, 16, d, dtype=torch.int8, device="cuda")
    assert kc.numel() > 2 ** 31
    ks = torch.full((nb, hkv), float("nan"), device="cuda")
    vs = ks.clone()
    lens, first = [70, 16, 33], nb - 9
    slots = torch.cat([torch.arange(n, device="cuda") + 16 * (first + o) for n, o in zip(lens, (0, 5, 6))])
    x = torch.randn(2, len(slots), hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_cache_write_scaled(x[0], x[1], slots, kc, vc, ks, vs, err)
    tables = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    for s, (n, o) in enumerate(zip(lens, (0, 5, 6))):
        m = -(-n // 16)
        tables[s, :m] = torch.arange(first + o, first + o + m, device="cuda")
    q = torch.randn(3, 16, d, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(pa.pa_decode_scaled_workspace_size(16, hkv, d), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scaled(q, kc, vc, ks, vs, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), 80, 0.09, out, ws, err)
    assert pa.pa_wait(err) == 0
    cut = lambda t: to_values(t[first:])
    ref, mass, reach = step_ops.decode_scaled(q.double().cpu().numpy(), cut(kc), cut(vc), ks[first:].cpu().numpy(),
                                              vs[first:].cpu().numpy(), tables.cpu().numpy() - first, lens, 0.09)
    far = np.abs(out.double().cpu().numpy() - ref) - step_ops.attention_bound(ref, mass, reach, (70, 2.0 ** -11, 6.0))
    assert (far <= 0).all()


@pytest.mark.gpu
def test_decode_flags_bad_inputs(pa):
    """Lengths and blocks outside their ranges are flagged; the other sequences are right."""
    torch = torch_mod()
    t = Decode(pa, "int8", 4, 2, 64, [50, 20, 64, 33], seed=3)
    lens = t.t[5].clone()
    lens[1] = -3
    t.call(lens=lens)
    assert pa.pa_wait(t.err) == pa.PA_DEVERR_CONTEXT_LEN
    t.check(np.array([0, 2, 3]))
    t.err.zero_()
    lens[1] = t.mb * 16 + 1
    t.call(lens=lens, max_context=t.mb * 16)
    assert pa.pa_wait(t.err) == pa.PA_DEVERR_CONTEXT_LEN
    t.check(np.array([0, 2, 3]))
    t.err.zero_()
    tables = t.t[4].clone()
    tables[2, 1], tables[2, 2] = -1, len(t.kp)
    t.call(tables=tables)
    assert pa.pa_wait(t.err) == pa.PA_DEVERR_BLOCK_ID
    t.check(np.array([0, 1, 3]))
    t.err.zero_()
    t.call()
    assert pa.pa_wait(t.err) == 0
    t.check()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_decode_in_graphs_that_share_a_workspace(pa, code):
    """Two captured calls on one workspace, replayed with other lengths; another stream."""
    torch = torch_mod()
    a = Decode(pa, code, 8, 2, 128, [300, 20, 900], seed=1)
    b = Decode(pa, code, 8, 2, 128, [5, 700], seed=2)
    b.ws = a.ws
    side = torch.cuda.Stream()
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            t.call()
        graphs.append(g)
    for cut in (0, 17, 3):
        for t in (a, b):
            t.lens = np.maximum(t.lens - cut, 0).astype(np.int32)
            t.t[5].copy_(torch.from_numpy(t.lens))
            for s, n in enumerate(t.lens):      # rows behind the new end are finite or junk: both unread
                t.blocks[s] = -(-int(n) // 16)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for t in (a, b):
            assert pa.pa_wait(t.err) == 0
            t.check()
    a.out.zero_()
    with torch.cuda.stream(side):
        a.call()
    a.call(stream=side)
    side.synchronize()
    a.check()


@pytest.mark.gpu
def test_a_context_of_2_31_tokens(pa):
    """One context of 2^31 - 1 tokens (every table entry names the same block): the line of items,
    the lengths and the last block's tail hold at the end of 32 bits."""
    torch = torch_mod()
    rng = np.random.default_rng(31)
    L, d, n = 2 ** 31 - 1, 64, 2 ** 27
    kc = torch.from_numpy(rng.integers(-127, 128, (1, 1, 16, d)).astype(np.int8)).cuda()
    vc = torch.from_numpy(rng.integers(-127, 128, (1, 1, 16, d)).astype(np.int8)).cuda()
    ks, vs = torch.full((1, 1), 2.0 ** -7, device="cuda"), torch.full((1, 1), 2.0 ** -6, device="cuda")
    q = torch.from_numpy(rng.standard_normal((1, 2, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    tables = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    lens, err = torch.tensor([L], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pa.pa_decode_scaled_workspace_size(2, 1, d), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scaled(q, kc, vc, ks, vs, tables, lens, L, 0.125, out, ws, err)
    assert pa.pa_wait(err) == 0
    k, v = kc.double().cpu().numpy()[0, 0] * 2.0 ** -7, vc.double().cpu().numpy()[0, 0] * 2.0 ** -6
    s = 0.125 * q.double().cpu().numpy()[0] @ k.T
    w = np.exp(s - s.max(1, keepdims=True)) * np.where(np.arange(16) < 15, n, n - 1)
    w /= w.sum(1, keepdims=True)
    # a warp of at least 148 x 12 adds n / 1776 blocks to its sums one after the other, each addition
    # off by 2^-24 of the sum: in the sum of the weights and in the weighted one; then the roundings
    # of the weights (f16) and the output (bf16), 2^-10 for the exponentials and scores
    tol = 2 * (n / 1776) * 2.0 ** -24 + 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -10
    far = np.abs(out.double().cpu().numpy()[0] - w @ v) - tol * (w @ np.abs(v))
    assert (far <= 0).all()


def tight_bound(t, ref, mass, reach, lost):
    """attention_bound, with `lost` of the row's largest weight p * value scale for each 16-bit weight
    below f16's normal numbers, times the largest code."""
    top = step_ops.largest_weight(t.q.double().numpy(), t.kp, t.ks, t.vs, t.tables, t.lens, t.scale)
    return (step_ops.attention_bound(ref, mass, reach, (0, 2.0 ** -11, 0.0))
            + t.lens[:, None, None] * lost * top * step_ops.TOP[t.code])


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_blocks_of_very_different_size_closely(pa, code, d):
    """Scales far apart within a sequence, within what 16-bit weights lose: 2^-25 of the
    row's largest weight each (f16's smallest step is 2^-24, and no reference point lies above
    the largest weight)."""
    torch = torch_mod()
    rng = np.random.default_rng(1)
    t = Decode(pa, code, 8, 2, d, [400, 37, 1200], seed=9, spread=0.5)
    live = ~np.isnan(t.ks)
    for s, lo, hi in ((t.vs, -40, 40), (t.ks, -30, 2)):
        s[live] *= 2.0 ** rng.integers(lo, hi, live.sum())
    t.t[2], t.t[3] = torch.from_numpy(t.ks).cuda(), torch.from_numpy(t.vs).cuda()
    t.call()
    assert pa.pa_wait(t.err) == 0
    ref, mass, reach = step_ops.decode_scaled(t.q.double().numpy(), t.kp, t.vp, t.ks, t.vs, t.tables, t.lens, t.scale)
    got, bound = t.out.double().cpu().numpy(), tight_bound(t, ref, mass, reach, 2.0 ** -25)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= bound).all()
    # the bound is tight enough to see two percent, in every sequence
    assert (np.abs(1.02 * ref - ref) > bound).any((1, 2)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("reach_down", [13, 16])
def test_decode_behind_a_key_that_outweighs_the_others(pa, code, d, reach_down):
    """One token has nearly all of the probability and a value of zero, under the same scale as
    the others' values: the row is what the other tokens add, 2^-18 to 2^-23 of that weight."""
    torch = torch_mod()
    rng = np.random.default_rng(reach_down)
    t = Decode(pa, code, 8, 2, d, [16, 32, 5, 250], seed=3)
    t.ks[:], t.vs[:], t.scale = 1.0, 0.5, 1.0
    t.kp[:] = np.where(np.isnan(t.kp), t.kp, 0.0)
    first = [int(b) for b in t.tables[:, 0]]
    for s, n in enumerate(t.lens):
        for j, b in enumerate(int(b) for b in t.tables[s][:-(-int(n) // 16)]):
            t.kp[b, :, :, 0] = -rng.integers(reach_down - 1, reach_down + 1, t.kp[b, :, :, 0].shape)
    t.kp[first, :, 0, 0] = 0.0
    t.vp[first, :, 0] = 0.0
    t.q[:] = 0.0
    t.q[..., 0] = 1.0
    c = lambda a: torch.from_numpy(a).cuda()
    t.t[:4] = [to_pool(t.kp, code), to_pool(t.vp, code), c(t.ks), c(t.vs)]
    t.qd = t.q.cuda()
    t.call()
    assert pa.pa_wait(t.err) == 0
    ref, mass, reach = step_ops.decode_scaled(t.q.double().numpy(), t.kp, t.vp, t.ks, t.vs, t.tables, t.lens, t.scale)
    got = t.out.double().cpu().numpy()
    # weights are kept to 2^-11, and below 2^-21 of the largest one to 2^-32 of it
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tight_bound(t, ref, mass, reach, 2.0 ** -32)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [-200, -140, -125, -100, -60])
def test_decode_value_scales_at_both_ends_of_their_range(pa, code, d, low):
    """A block of zeros (its scale is the smallest, 2^-64) with one head's largest scores, and a
    block of values near 2^100 that the head gives 2^low of them and the other heads most: as
    the append leaves both."""
    torch = torch_mod()
    hkv, nb, L = 1, 4, 40
    q = torch.zeros(1, 4, d, dtype=torch.bfloat16)
    for h in range(4):
        q[0, h, h] = 1.0
    k = np.zeros((L, hkv, d))
    # natural units: a difference of `low` powers of two
    k[16:32, 0, 0] = np.round(low * np.log(2))
    k[16:32, 0, 1] = 40.0
    v = np.zeros((L, hkv, d))
    rng = np.random.default_rng(-low)
    v[16:32] = rng.standard_normal((16, hkv, d)) * 2.0 ** 100
    kb, vb = bf16(k), bf16(v)
    slots = np.array([2, 0, 3])[np.arange(L) // 16] * 16 + np.arange(L) % 16
    kp = np.zeros((nb, hkv, 16, d))
    sc = np.full((nb, hkv), np.nan, np.float32)
    got, flag = check_write(pa, kb, vb, slots, kp, kp, sc, sc, code)
    assert flag == 0 and got[3][2, 0] == 2.0 ** -64 and got[3][0, 0] > 2.0 ** 90
    tables, lens = np.array([[2, 0, 3]], np.int32), np.array([L], np.int32)
    S = 3000         # the same sequence over and over: a warp has several blocks in a row
    c = lambda a: torch.from_numpy(a).cuda()
    out, err = torch.empty(S, 4, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_decode_scaled_workspace_size(4, 1, d), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scaled(c(q.float().numpy().repeat(S, 0)).to(torch.bfloat16), to_pool(got[0], code), to_pool(got[1], code), c(got[2]),
                        c(got[3]), c(tables.repeat(S, 0)), c(lens.repeat(S)), 48, 1.0, out, ws, err)
    assert pa.pa_wait(err) == 0
    qq = q.double().numpy()
    ref, mass, reach = step_ops.decode_scaled(qq, *got, tables, lens, 1.0)
    top = step_ops.largest_weight(qq, got[0], got[2], got[3], tables, lens, 1.0)
    bound = step_ops.attention_bound(ref, mass, reach, (0, 2.0 ** -11, 0.0)) + L * 2.0 ** -25 * top * step_ops.TOP[code]
    g = out.double().cpu().numpy()
    assert np.isfinite(g).all() and (np.abs(g - ref) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_append_of_rows_beyond_32_bits(pa, code):
    """Rows of a fused projection of more than 2^32 bytes, the last tokens in blocks of their own (the
    others are padding)."""
    torch = torch_mod()
    H, d, T, n = 8, 128, 240_000, 70
    rng = np.random.default_rng(12)
    x = torch.zeros(T, 10 * H, d, dtype=torch.bfloat16, device="cuda")
    assert x.numel() * 2 > 2 ** 32
    x[-n:] = bf16(rng.standard_normal((n, 10 * H, d))).cuda()
    k, v = x[:, 8 * H:9 * H], x[:, 9 * H:]
    kp, ks = random_pool(rng, 9, H, d, code)
    slots = np.full(T, -1, np.int64)
    slots[-n:] = appended(rng, 9, [5, 30], (20, 50))
    got, flag = run_write(pa, k, v, slots, kp, kp, ks, ks, code)
    assert flag == 0
    want = [kp.copy(), kp.copy(), ks.copy(), ks.copy()]
    for rows, i in ((k, 0), (v, 1)):
        step_ops.cache_write_scaled(rows[-n:].double().cpu().numpy(), slots[-n:], want[i], want[2 + i], code)
    assert all(same(g, w) for g, w in zip(got, want))


@pytest.mark.gpu
def test_decode_of_16384_sequences(pa):
    """The most sequences a call takes, short and long contexts among them."""
    rng = np.random.default_rng(16)
    lens = rng.integers(0, 20, 16384)
    lens[rng.integers(0, 16384, 30)] = rng.integers(500, 900, 30)
    t = Decode(pa, "e4m3", 2, 1, 64, lens, seed=16)
    t.call()
    assert pa.pa_wait(t.err) == 0
    t.check(np.concatenate([np.nonzero(lens > 100)[0], np.arange(40), rng.integers(0, 16384, 200), np.arange(16340, 16384)]))
