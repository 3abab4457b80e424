"""The serving-step operators as they are used together: plan on the GPU, attention over
packed prompts, append into the 8-bit cache, decode steps, release -- all device-side
state, against fp64; and PagedKVCache with a scale per block."""
import numpy as np
import pytest

from oracle import step_ops
from test_gpu_scaled_cache import CODES, code_dtype, to_values, torch_mod

pytestmark = pytest.mark.gpu


def rows(rng, T, h, d):
    torch = torch_mod()
    return torch.from_numpy(rng.standard_normal((T, h, d)).astype(np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def within(got, ref, mass, reach, tokens):
    far = np.abs(got - ref) - step_ops.attention_bound(ref, mass, reach, tokens)
    assert np.isfinite(got).all() and (far <= 0).all(), f"off by {far.max():.3g} more than the bound"


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_prompts_then_decode_steps(pa, code, hq, hkv, d):
    torch = torch_mod()
    rng = np.random.default_rng(hq)
    S, N, mb, cap = 7, 120, 12, 600
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device="cuda")
    order = rng.permutation(N).astype(np.int32)
    lens, tables, nf, err = z(S), torch.full((S, mb), -1, dtype=torch.int32, device="cuda"), z(1) + N, z(1)
    free, slots, starts = torch.from_numpy(order).cuda(), z(cap, dt=torch.int64), z(S + 1)
    kc, vc = torch.zeros(2, N, hkv, 16, d, device="cuda").to(code_dtype(code)).unbind(0)
    kc, vc = kc.contiguous(), vc.contiguous()
    ks, vs = torch.full((2, N, hkv), float("nan"), device="cuda").unbind(0)
    ks, vs = ks.contiguous(), vs.contiguous()
    kref, vref = np.zeros((N, hkv, 16, d)), np.zeros((N, hkv, 16, d))
    ksref, vsref = np.full((N, hkv), np.nan), np.full((N, hkv), np.nan)
    ws = torch.empty(max(pa.pa_decode_scaled_workspace_size(hq, hkv, d),
                         pa.pa_prefill_packed_workspace_size(cap, S, hq, hkv)), dtype=torch.uint8, device="cuda")
    scale = d ** -0.5
    counts = [40, 1, 17, 0, 128, 16, 33]
    for step in range(6):
        c = torch.tensor(counts, dtype=torch.int32, device="cuda")
        ref = step_ops.step_plan(np.array(counts), lens.cpu().numpy(), tables.cpu().numpy(), free.cpu().numpy(), int(nf), cap)
        pa.pa_step_plan(c, lens, tables, free, nf, slots, starts, err_flag=err)
        assert np.array_equal(tables.cpu().numpy(), ref[0]) and np.array_equal(slots.cpu().numpy(), ref[1])
        T = cap   # the whole padded buffer, as a captured step would pass it
        fused = rows(rng, T, hq + 2 * hkv, d)
        q, k, v = fused.split([hq, hkv, hkv], 1)
        if step == 0:
            out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
            pa.pa_prefill_packed(q, k, v, starts, 128, scale, out, ws, err)
            o, mass, reach = step_ops.packed_attention(f64(q), f64(k), f64(v), ref[2], scale)
            n = int(ref[2][-1])
            within(f64(out)[:n], o[:n], mass[:n], reach[:n], (0, 2.0 ** -8, 0.0))
            assert (out[n:] == 7).all()
        pa.pa_cache_write_scaled(k, v, slots, kc, vc, ks, vs, err)
        step_ops.cache_write_scaled(f64(k), ref[1], kref, ksref, code)
        step_ops.cache_write_scaled(f64(v), ref[1], vref, vsref, code)
        assert np.array_equal(to_values(kc), kref) and np.array_equal(to_values(vc), vref)
        assert np.array_equal(ks.cpu().numpy(), ksref, equal_nan=True) and np.array_equal(vs.cpu().numpy(), vsref, equal_nan=True)
        qd = rows(rng, S, hq, d)
        out = torch.empty_like(qd)
        pa.pa_decode_scaled(qd, kc, vc, ks, vs, tables, lens, mb * 16, scale, out, ws, err)
        o, mass, reach = step_ops.decode_scaled(f64(qd), kref, vref, ksref, vsref, ref[0], ref[3], scale)
        within(f64(out), o, mass, reach, (mb * 16, 2.0 ** -11, 6.0))
        if step == 3:
            done = torch.tensor([0, 1, 0, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
            pa.pa_step_release(done, lens, tables, free, nf, err_flag=err)
            assert lens[1] == 0 and lens[4] == 0 and (tables[4] == -1).all()
        counts = [1, 1, 1, 0, 1, 1, 1] if step != 3 else [1, 20, 1, 3, 50, 1, 1]
    assert pa.pa_wait(err) == 0


@pytest.mark.parametrize("code", CODES)
def test_paged_cache_with_block_scales(pa, code):
    """Prompts, a fork with copy on write, and decode steps through PagedKVCache."""
    from paged_kv_cache_389_b200.cache import PagedKVCache
    torch = torch_mod()
    rng = np.random.default_rng(3)
    hq, hkv, d, scale = 8, 4, 64, 0.125
    kv = PagedKVCache(64, hkv, d, code_dtype(code), block_scales=True)
    assert kv.key_scales.shape == (64, hkv) and torch.isnan(kv.key_scales).all()
    for s in (0, 1):
        kv.add_seq(s)
    counts = [37, 60]
    q, k, v = rows(rng, 97, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    out = kv.prompt(q, k, v, [0, 1], counts, scale)
    o, mass, reach = step_ops.packed_attention(f64(q), f64(k), f64(v), np.array([0, 37, 97]), scale)
    within(f64(out), o, mass, reach, (0, 2.0 ** -8, 0.0))
    with pytest.raises(ValueError):
        kv.prompt(q, k, v, [0, 1], counts, scale)
    with pytest.raises(ValueError):
        kv.append([0, 1, 0], k[:3], v[:3])
    with pytest.raises(ValueError):
        kv.prefill(q[:2].unsqueeze(1), [0, 1], [1, 1], scale)
    kv.fork(0, 2)
    for _ in range(3):
        kn, vn, qn = rows(rng, 3, hkv, d), rows(rng, 3, hkv, d), rows(rng, 3, hq, d)
        slots, pairs = kv.append([0, 1, 2], kn, vn)
        got = kv.decode(qn, [0, 1, 2], scale)
        t, l = kv.manager.build_tables([0, 1, 2], 8)
        o, mass, reach = step_ops.decode_scaled(f64(qn), to_values(kv.key_cache), to_values(kv.value_cache),
                                                kv.key_scales.cpu().numpy(), kv.value_scales.cpu().numpy(), t, l, scale)
        within(f64(got), o, mass, reach, (64, 2.0 ** -11, 6.0))
    # what the cache holds is what was appended, to half a step of each block's scale
    b = kv.manager.block_table(0)
    held = np.concatenate([to_values(kv.key_cache[x:x + 1])[0] * kv.key_scales[x].cpu().numpy()[:, None, None] for x in b[:2]], 1)
    kk = f64(k)[:32].transpose(1, 0, 2)
    step = np.repeat(np.stack([kv.key_scales[x].cpu().numpy() for x in b[:2]], 1), 16, 1)[:, :, None]
    half = 0.5 * step if code == "int8" else np.maximum(2.0 ** -4 * np.abs(kk), 2.0 ** -10 * step)
    assert (np.abs(held - kk) <= half).all()
    assert pa.pa_wait(kv.err_flag) == 0


def test_prompt_on_a_bf16_cache(pa):
    """prompt() over a bf16 pool: the same attention as the chunked prefill of the same tokens."""
    from paged_kv_cache_389_b200.cache import PagedKVCache
    torch = torch_mod()
    rng = np.random.default_rng(5)
    kv = PagedKVCache(64, 2, 128, torch.bfloat16)
    kv.add_seq(0)
    kv.add_seq(1)
    q, k, v = rows(rng, 150, 12, 128).split([8, 2, 2], 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = kv.prompt(q, k, v, [0, 1], [100, 50], 0.09, stream=side)
    side.synchronize()
    padded = torch.zeros(2, 100, 8, 128, dtype=torch.bfloat16, device="cuda")
    padded[0], padded[1, :50] = q[:100], q[100:]
    chunk = kv.prefill(padded, [0, 1], [100, 50], 0.09)
    # both are off by at most their own rounding and that of P (2^-8 each) of the same attention
    o, mass, reach = step_ops.packed_attention(f64(q), f64(k), f64(v), np.array([0, 100, 150]), 0.09)
    within(f64(out), o, mass, reach, (0, 2.0 ** -8, 0.0))
    within(np.concatenate([f64(chunk[0]), f64(chunk[1, :50])]), o, mass, reach, (0, 2.0 ** -8, 0.0))
    assert pa.pa_wait(kv.err_flag) == 0


def test_prompt_refusals_leave_the_manager_alone(pa):
    from paged_kv_cache_389_b200.cache import PagedKVCache
    torch = torch_mod()
    rng = np.random.default_rng(1)
    kv = PagedKVCache(8, 2, 64, torch.int8, block_scales=True)
    for s in (0, 1):
        kv.add_seq(s)
    q, k, v = rows(rng, 40, 8, 64).split([4, 2, 2], 1)
    for seqs, counts in (([0, 0], [20, 20]), ([0, 1], [20, 21]), ([0, 1], [40]), ([0, 1], [50, -10])):
        with pytest.raises(ValueError):
            kv.prompt(q, k, v, seqs, counts, 0.1)
    with pytest.raises(pa.PAError):    # six query heads on two kv heads: no group of three
        kv.prompt(rows(rng, 40, 6, 64), k, v, [0, 1], [20, 20], 0.1)
    big = rows(rng, 200, 8, 64)
    with pytest.raises(pa.PAError):    # 13 blocks of a pool of 8
        kv.prompt(*big.split([4, 2, 2], 1), [0, 1], [100, 100], 0.1)
    assert kv.manager.num_tokens(0) == 0 and kv.manager.num_tokens(1) == 0 and kv.manager.num_free() == 8
    with pytest.raises(ValueError):
        PagedKVCache(8, 2, 64, torch.float32).prompt(q, k, v, [], [], 0.1)
    kv.prompt(q[:0], k[:0], v[:0], [0, 1], [0, 0], 0.1)
    assert pa.pa_wait(kv.err_flag) == 0


def test_calls_on_a_stream_of_their_own(pa):
    """Prompts, appends and decodes through PagedKVCache on a side stream while the current one
    allocates and overwrites: nothing a call made for itself is taken from under it."""
    from paged_kv_cache_389_b200.cache import PagedKVCache
    torch = torch_mod()
    rng = np.random.default_rng(8)
    fused, qn = rows(rng, 500, 8, 64), rows(rng, 2, 4, 64)
    q, k, v = fused.split([4, 2, 2], 1)
    results = []
    for side in (None, torch.cuda.Stream()):
        kv = PagedKVCache(64, 2, 64, torch.float8_e4m3fn, block_scales=True)
        kv.add_seq(0)
        kv.add_seq(1)
        torch.cuda.synchronize()
        outs = [kv.prompt(q, k, v, [0, 1], [300, 200], 0.1, stream=side)]
        for i in range(8):
            kv.append([0, 1], k[i:i + 2], v[i:i + 2], stream=side)
            outs.append(kv.decode(qn, [0, 1], 0.1, stream=side))
            for n in (4, 8, 64, 4096, 1 << 20):    # the sizes of the calls' own tensors
                torch.full((n,), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert int(kv.err_flag) == 0
        results.append(outs)
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("code", CODES)
def test_captured_steps_follow_the_device(pa, code):
    """A prompt step and a decode step, each captured once (with one workspace between them) on a
    side stream and replayed with other counts, rows and finished sequences, against the same
    steps called one by one: every table, slot, code, scale and output the same, bit for bit."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    hq, hkv, d, S, N, mb, cap = 8, 2, 128, 5, 96, 20, 500
    order = torch.from_numpy(rng.permutation(N).astype(np.int32)).cuda()

    class State:
        def __init__(self):
            z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device="cuda")
            self.counts, self.done, self.lens, self.nf, self.err = z(S), z(S), z(S), z(1) + N, z(1)
            self.tables, self.free = z(S, mb) - 1, order.clone()
            self.slots, self.starts = z(cap, dt=torch.int64), z(S + 1)
            self.kc, self.vc = (torch.zeros(N, hkv, 16, d, device="cuda").to(code_dtype(code)) for _ in range(2))
            self.ks, self.vs = (torch.full((N, hkv), float("nan"), device="cuda") for _ in range(2))
            self.x, self.q = rows(rng, cap, hq + 2 * hkv, d), rows(rng, S, hq, d)
            self.out, self.dec = torch.zeros(cap, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(self.q)
            self.ws = torch.empty(max(pa.pa_decode_scaled_workspace_size(hq, hkv, d),
                                      pa.pa_prefill_packed_workspace_size(cap, S, hq, hkv)), dtype=torch.uint8, device="cuda")

        def step(self, prompts):
            q, k, v = self.x.split([hq, hkv, hkv], 1)
            pa.pa_step_release(self.done, self.lens, self.tables, self.free, self.nf, err_flag=self.err)
            pa.pa_step_plan(self.counts, self.lens, self.tables, self.free, self.nf, self.slots, self.starts, err_flag=self.err)
            if prompts:
                pa.pa_prefill_packed(q, k, v, self.starts, 300, 0.09, self.out, self.ws, self.err)
            pa.pa_cache_write_scaled(k, v, self.slots, self.kc, self.vc, self.ks, self.vs, self.err)
            pa.pa_decode_scaled(self.q, self.kc, self.vc, self.ks, self.vs, self.tables, self.lens, mb * 16, 0.09, self.dec,
                                self.ws, self.err)

    twin, state = State(), State()
    scratch = State()
    for prompts in (True, False):        # libraries and attributes set up before the capture
        scratch.step(prompts)
    torch.cuda.synchronize()
    graphs = {}
    side = torch.cuda.Stream()
    for prompts in (True, False):
        graphs[prompts] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[prompts], stream=side):
            state.step(prompts)
    for prompts, counts, done in ((True, [33, 1, 300, 0, 16], [0, 0, 0, 0, 0]), (False, [1, 1, 1, 0, 1], [0, 0, 0, 0, 0]),
                                  (False, [1, 1, 1, 0, 1], [0, 0, 0, 0, 0]), (True, [0, 0, 250, 190, 0], [0, 0, 1, 0, 0]),
                                  (False, [1, 1, 1, 1, 1], [0, 1, 0, 0, 0]), (False, [5, 0, 2, 1, 20], [0, 0, 0, 0, 0])):
        x, q = rows(rng, cap, hq + 2 * hkv, d), rows(rng, S, hq, d)
        for s in (twin, state):
            s.counts.copy_(torch.tensor(counts))
            s.done.copy_(torch.tensor(done))
            s.x.copy_(x)
            s.q.copy_(q)
        twin.step(prompts)
        graphs[prompts].replay()
        torch.cuda.synchronize()
        assert int(twin.err) == 0 and int(state.err) == 0
        T = int(twin.starts[-1])
        assert T == sum(counts)
        for name in ("lens", "nf", "tables", "free", "slots", "starts", "dec"):
            assert torch.equal(getattr(twin, name), getattr(state, name)), name
        if prompts:
            assert torch.equal(twin.out[:T], state.out[:T])
        for name in ("kc", "vc"):
            assert torch.equal(getattr(twin, name).view(torch.uint8), getattr(state, name).view(torch.uint8)), name
        for name in ("ks", "vs"):
            assert torch.equal(getattr(twin, name).nan_to_num(7), getattr(state, name).nan_to_num(7)), name


def test_calls_that_overlap(pa):
    """Packed attention and 8-bit decodes on three streams at once, each with a workspace of its
    own: the results of the same calls one after the other, bit for bit."""
    torch = torch_mod()
    rng = np.random.default_rng(33)
    hq, hkv, d, S = 8, 2, 64, 40
    n = rng.integers(1, 700, S)
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    T = int(starts[-1])
    q, k, v = rows(rng, T, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    blocks = -(-n // 16)
    N = int(blocks.sum())
    tables = np.full((S, int(blocks.max())), -1, np.int32)
    ids, at = rng.permutation(N), 0
    for s in range(S):
        tables[s, :blocks[s]] = ids[at:at + blocks[s]]
        at += blocks[s]
    slots = np.concatenate([tables[s, np.arange(n[s]) // 16].astype(np.int64) * 16 + np.arange(n[s]) % 16 for s in range(S)])
    tables, lens = torch.from_numpy(tables).cuda(), torch.from_numpy(n.astype(np.int32)).cuda()
    kc, vc = (torch.zeros(N, hkv, 16, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(N, hkv, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_cache_write_scaled(k, v, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, err)
    qd = rows(rng, S, hq, d)

    def attend(stream, out, ws):
        pa.pa_prefill_packed(q, k, v, starts, 700, 0.125, out, ws, err, stream)

    def decode(stream, out, ws):
        pa.pa_decode_scaled(qd, kc, vc, ks, vs, tables, lens, int(n.max()), 0.125, out, ws, err, stream)

    size = max(pa.pa_prefill_packed_workspace_size(T, S, hq, hkv), pa.pa_decode_scaled_workspace_size(hq, hkv, d))
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    want = torch.zeros_like(q.contiguous()), torch.zeros_like(qd)
    attend(None, want[0], ws[0])
    decode(None, want[1], ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        got = [torch.zeros_like(want[0]), torch.zeros_like(want[1]), torch.zeros_like(want[1])]
        torch.cuda.synchronize()
        for _ in range(4):
            for call, stream, out, w in zip((attend, decode, decode), streams, got, ws):
                call(stream, out, w)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[1])
    assert int(err) == 0


def test_prompt_refuses_what_the_write_would(pa):
    """What the append would refuse -- rows of another head_dim or head count than the pool's, a
    pool it cannot write -- prompt() refuses before the manager hands out blocks."""
    from paged_kv_cache_389_b200.cache import PagedKVCache
    torch = torch_mod()
    rng = np.random.default_rng(2)
    e4m3 = torch.float8_e4m3fn
    pools = [PagedKVCache(8, 2, 128, torch.int8, block_scales=True), PagedKVCache(8, 2, 128, e4m3, block_scales=True),
             PagedKVCache(8, 2, 128, torch.bfloat16), PagedKVCache(8, 2, 128, e4m3),
             PagedKVCache(8, 2, 64, e4m3),                       # one scale: written at head_dim 128 only
             PagedKVCache(8, 2, 128, e4m3, k_scale=0.0)]
    wrong = [[(4, 2, 64), (4, 1, 128), (4, 4, 128)]] * 4 + [[(4, 2, 64)], [(4, 2, 128)]]
    for kv, shapes in zip(pools, wrong):
        kv.add_seq(0)
        for hq, hkv, d in shapes:
            q, k, v = rows(rng, 40, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
            with pytest.raises((ValueError, AssertionError, pa.PAError)):
                kv.prompt(q, k, v, [0], [40], 0.1)
            assert kv.manager.num_tokens(0) == 0 and kv.manager.num_free() == 8
    for kv in pools[:4]:                                         # and is none the worse for it
        q, k, v = rows(rng, 40, 8, 128).split([4, 2, 2], 1)
        out = kv.prompt(q, k, v, [0], [40], 0.1)
        o, mass, reach = step_ops.packed_attention(f64(q), f64(k), f64(v), np.array([0, 40]), 0.1)
        within(f64(out), o, mass, reach, (0, 2.0 ** -8, 0.0))
        assert kv.manager.num_tokens(0) == 40 and pa.pa_wait(kv.err_flag) == 0
