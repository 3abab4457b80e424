"""Causal attention over packed prompts against the fp64 definition, and its refusals."""
import ctypes as C

import numpy as np
import pytest

from oracle import step_ops
from test_abi import _gpu_visible


def torch_mod():
    import torch
    return torch


@pytest.mark.skipif(_gpu_visible(), reason="passes placeholder device addresses: only where no GPU is reachable")
def test_host_validation(pa):
    L, p, odd = pa._lib, C.c_void_p(0x10000), C.c_void_p(0x10008)
    need = pa.pa_prefill_packed_workspace_size(100, 3, 8, 2)
    f = lambda q=p, k=p, v=p, qs=1024, ks=256, vs=256, st=p, S=3, T=100, ml=60, hq=8, hkv=2, d=128, ws=p, wsb=need, out=p: \
        L.pa_prefill_packed(q, k, v, qs, ks, vs, st, S, T, ml, hq, hkv, d, 0.1, ws, wsb, out, None, None)
    bad, uns = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(q=odd), dict(k=odd), dict(v=odd), dict(out=odd), dict(ws=odd),
               dict(ws=None), dict(wsb=need - 1), dict(st=None), dict(S=-1), dict(T=-1), dict(ml=-1), dict(qs=1016), dict(ks=255),
               dict(vs=260), dict(hkv=0), dict(hq=0), dict(hq=7)):
        assert f(**kw) == bad, kw
    for kw in (dict(d=96), dict(d=256), dict(hq=32, qs=4096), dict(S=16385, wsb=1 << 30)):
        assert f(**kw) == uns, kw
    for kw in (dict(S=0), dict(T=0), dict(ml=0)):
        assert f(**kw) == pa.PA_OK, kw
    assert pa.pa_prefill_packed_workspace_size(100, 3, 7, 2) == 0
    assert need == 16 + (100 * 4 // 256 + 3) * 16


def test_binding_refuses_wrong_tensors(pa):
    torch = torch_mod()
    q, k = torch.zeros(9, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    st, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    for a in ((q.float(), k, k, st), (q, k[:8], k, st), (q, k, k.float(), st), (q, k, k, st.long()), (q, k[:, :, ::2], k, st),
              (q, k, k, st)):           # the last: right, but not on a GPU
        with pytest.raises((AssertionError, ValueError)):
            pa.pa_prefill_packed(*a[:3], a[3], 5, 0.1, torch.empty_like(q), ws)


def bf16(x):
    torch = torch_mod()
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def inputs(rng, T, hq, hkv, d, fused):
    torch = torch_mod()
    if fused:
        x = bf16(rng.standard_normal((T, hq + 2 * hkv, d))).cuda()
        return x.split([hq, hkv, hkv], 1)
    return tuple(bf16(rng.standard_normal((T, h, d))).cuda() for h in (hq, hkv, hkv))


def run(pa, q, k, v, starts, scale, max_len=None, out=None, ws=None, stream=None):
    torch = torch_mod()
    T, hq, d = q.shape
    starts = np.asarray(starts, np.int32)
    st = torch.from_numpy(starts).cuda()
    out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    n = pa.pa_prefill_packed_workspace_size(T, len(starts) - 1, hq, k.shape[1])
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_len = int(max(np.diff(starts).max(initial=1), 1)) if max_len is None else max_len
    pa.pa_prefill_packed(q, k, v, st, max_len, scale, out, ws, err, stream)
    return out, pa.pa_wait(err, stream)


def check(got, q, k, v, starts, scale):
    f = lambda t: t.double().cpu().numpy()
    ref, mass, reach = step_ops.packed_attention(f(q), f(k), f(v), starts, scale)
    rows = np.zeros(len(ref), bool)
    for a, b in zip(starts[:-1], starts[1:]):
        rows[a:b] = True
    g = f(got)
    assert (g[~rows] == 7).all()              # rows of no sequence are left alone
    # P is rounded to bf16 (2^-8)
    bound = step_ops.attention_bound(ref, mass, reach, (0, 2.0 ** -8, 0.0))
    far = (np.abs(g - ref) - bound)[rows]
    assert np.isfinite(g[rows]).all() and (far <= 0).all(), f"off by {far.max():.3g} more than the bound"


CASES = [
    ((0, 1), 0), ((0, 5), 3), ((0, 128), 0), ((0, 129), 1), ((0, 300), 0), ((0, 1, 2, 3, 40, 40, 41), 2), ((3, 3, 20, 148, 149, 406), 9),
    ((0, 64, 128, 192, 256, 320), 0), ((0, 700, 701, 1900), 0), (tuple(range(0, 200, 7)), 5), ((0, 0), 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (2, 2, 64), (4, 2, 128), (8, 2, 64), (8, 1, 128), (12, 3, 128), (16, 2, 64), (2, 1, 64)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_packed_matches_the_definition(pa, hq, hkv, d, case):
    starts, behind = CASES[case]
    rng = np.random.default_rng(case * 10 + hq + d)
    T = starts[-1] + behind
    if T == 0:
        pytest.skip("no rows")
    q, k, v = inputs(rng, T, hq, hkv, d, fused=case % 2 == 0)
    out, flag = run(pa, q, k, v, starts, d ** -0.5)
    assert flag == 0
    check(out, q, k, v, np.array(starts), d ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.11, 0.9])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(pa, scale, d):
    """A zero scale (the mean of the values so far), a negative one, one that makes the
    softmax nearly one-hot and moves the reference point often."""
    rng = np.random.default_rng(3)
    starts = np.array([0, 200, 611])
    q, k, v = inputs(rng, 611, 4, 1, d, True)
    out, flag = run(pa, q, k, v, starts, scale)
    assert flag == 0
    check(out, q, k, v, starts, scale)


@pytest.mark.gpu
def test_growing_scores_move_the_reference(pa):
    """Keys that grow along the sequence: every tile raises the maxima by far."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    q, k, v = inputs(rng, 900, 2, 1, 128, False)
    k = (k.float() * torch.linspace(0.1, 30, 900, device="cuda")[:, None, None]).to(torch.bfloat16)
    out, flag = run(pa, q, k, v, [0, 900], 0.5)
    assert flag == 0
    check(out, q, k, v, np.array([0, 900]), 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (2, 2, 64), (8, 1, 64)])
def test_what_is_masked_never_reaches_a_row(pa, hq, hkv, d):
    """Infinities and NaN in later keys and values, in the next sequence and behind the last."""
    torch = torch_mod()
    rng = np.random.default_rng(7)
    starts = np.array([0, 150, 150, 470])
    q, k, v = inputs(rng, 500, hq, hkv, d, False)
    clean = run(pa, q, k, v, starts, 0.1)[0].clone()
    for bad_k, bad_v in ((float("nan"), float("nan")), (float("inf"), float("-inf")), (1e38, float("nan")), (0.0, float("inf"))):
        for at in (slice(149, 150), slice(400, 470), slice(333, 334), slice(470, 500)):
            k2, v2 = k.clone(), v.clone()
            k2[at], v2[at] = bad_k, bad_v
            out, flag = run(pa, q, k2, v2, starts, 0.1)
            assert flag == 0
            # rows in front of the bad ones, and the other sequences, as without them
            seq = (starts[:-1][starts[:-1] <= at.start].max(), min([s for s in starts if s > at.start], default=500))
            same = [i for i in range(470) if i < at.start or i >= seq[1]]
            ref, mass, reach = step_ops.packed_attention(*(x.double().cpu().numpy() for x in (q, k, v)), starts, 0.1)
            bound = step_ops.attention_bound(ref, mass, reach, (0, 2.0 ** -8, 0.0))
            g = out.double().cpu().numpy()
            assert (np.abs(g - ref) <= bound)[same].all()
            if at.start < 470 and bad_v != bad_v:
                assert np.isnan(g[at.start]).any()
    assert torch.isfinite(clean.float()).all()


@pytest.mark.gpu
def test_bad_starts_are_flagged(pa):
    torch = torch_mod()
    rng = np.random.default_rng(9)
    q, k, v = inputs(rng, 300, 4, 2, 64, True)
    for starts, max_len, good in (((0, 100, 90, 300), 250, [(0, 100)]), ((-5, 100, 200), 200, [(100, 200)]),
                                  ((0, 100, 301), 201, [(0, 100)]), ((0, 100, 300), 120, [(0, 100)])):
        out, flag = run(pa, q, k, v, starts, 0.1, max_len)
        assert flag == pa.PA_DEVERR_CHUNK, starts
        a, b = good[0]
        only = out.clone()
        only[:a], only[b:] = 7, 7
        if starts == (0, 100, 90, 300):
            # rows 90 .. 99 are also the first ones of the (valid) third sequence: both write them
            only = only[:90]
            check(only, q[:90], k[:90], v[:90], np.array([0, 90]), 0.1)
            continue
        check(only, q, k, v, np.array([a, b]), 0.1)
    out, flag = run(pa, q, k, v, (0, 100, 300), 0.1)
    assert flag == 0
    check(out, q, k, v, np.array([0, 100, 300]), 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 1, 128), (8, 2, 64)])
@pytest.mark.parametrize("seqs", [40, 3000])
def test_short_sequences_without_a_list(pa, hq, hkv, d, seqs):
    """Sequences of at most one pair of row tiles (empty ones and the longest among them), few
    enough to be taken in turn and too many for that; then with bad ones between them."""
    torch = torch_mod()
    rng = np.random.default_rng(hq + d)
    most = 256 // (hq // hkv)
    n = rng.integers(0, most if seqs < 100 else 6, seqs, endpoint=True)
    n[3], n[7], n[-1] = most, 0, 1
    starts = np.concatenate([[2], 2 + np.cumsum(n)])
    q, k, v = inputs(rng, int(starts[-1]) + 3, hq, hkv, d, True)
    out, flag = run(pa, q, k, v, starts, 0.11, most)
    assert flag == 0
    check(out, q, k, v, starts, 0.11)
    # sequences of that length (the fourth, and any other) are longer than announced: left out
    full = run(pa, q, k, v, starts, 0.11, most)[0]
    out, flag = run(pa, q, k, v, starts, 0.11, most - 1)
    assert flag == pa.PA_DEVERR_CHUNK
    for s in np.nonzero(n == most)[0]:
        assert (out[starts[s]:starts[s + 1]] == 7).all()
        out[starts[s]:starts[s + 1]] = full[starts[s]:starts[s + 1]]
    check(out, q, k, v, starts, 0.11)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [2000, 4000])
def test_a_stream_far_behind_the_other(pa, seqs):
    """Rows that are computed again (masked infinities) keep one stream of a CTA busy while the
    other goes through dozens of short sequences: their records have to wait for the slow one."""
    rng = np.random.default_rng(4)
    n = np.concatenate([[256] * 8, rng.integers(1, 4, seqs - 8)])
    starts = np.concatenate([[0], np.cumsum(n)])
    q, k, v = inputs(rng, int(starts[-1]), 1, 1, 64, False)
    v[starts[1:9] - 1] = float("inf")     # seen by the last row only
    out, flag = run(pa, q, k, v, starts, 0.125)
    assert flag == 0
    assert np.isinf(out[starts[1:9] - 1].double().cpu().numpy()).all()
    out[starts[1:9] - 1] = 0
    v[starts[1:9] - 1] = 0
    mask = np.zeros(len(q), bool)
    mask[starts[1:9] - 1] = True
    f = lambda x: x.double().cpu().numpy()
    o, mass, reach = step_ops.packed_attention(f(q), f(k), f(v), starts, 0.125)
    far = np.abs(f(out) - o) - step_ops.attention_bound(o, mass, reach, (0, 2.0 ** -8, 0.0))
    assert (far[~mask] <= 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,seqs,hq", [(300, 40, 4), (32 * (2 ** 19 + 1), 16384, 8)])
def test_starts_that_go_back_and_forth_list_nothing(pa, tokens, seqs, hq):
    """Starts 0, T, 0, T, ...: every second sequence is all of the rows.  Their pairs do not fit
    the list, also where 32-bit sums of them would come round to a small number (the second
    case: 8192 x (2^19 + 1) = 2^32 + 8192): flagged, and no row is written."""
    torch = torch_mod()
    z = lambda h: torch.empty(tokens, h, 64, dtype=torch.bfloat16, device="cuda")
    q, k, v, out = z(hq), z(1), z(1), z(hq).fill_(7)
    starts = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = tokens
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_prefill_packed_workspace_size(tokens, seqs, hq, 1), dtype=torch.uint8, device="cuda")
    pa.pa_prefill_packed(q, k, v, starts, tokens, 0.1, out, ws, err)
    assert pa.pa_wait(err) == pa.PA_DEVERR_CHUNK
    assert (out[::101] == 7).all() and (out[-300:] == 7).all()


@pytest.mark.gpu
def test_many_sequences_and_a_long_one(pa):
    rng = np.random.default_rng(12)
    starts = np.concatenate([[0], np.cumsum(rng.integers(0, 9, 3000))])
    q, k, v = inputs(rng, int(starts[-1]), 2, 1, 64, True)
    out, flag = run(pa, q, k, v, starts, 0.125)
    assert flag == 0
    check(out, q, k, v, starts, 0.125)
    q, k, v = inputs(rng, 5000, 1, 1, 128, False)
    out, flag = run(pa, q, k, v, [0, 5000], 0.09)
    assert flag == 0
    check(out, q, k, v, np.array([0, 5000]), 0.09)


@pytest.mark.gpu
def test_in_graphs_that_share_a_workspace_and_on_another_stream(pa):
    torch = torch_mod()
    rng = np.random.default_rng(1)
    side, graphs = torch.cuda.Stream(), []
    ws = torch.full((4096,), 0xFF, dtype=torch.uint8, device="cuda")
    for hq, hkv, d, cuts in ((4, 1, 128, [(0, 300, 500), (0, 10, 500), (5, 5, 499)]), (2, 2, 64, [(0, 500, 500), (7, 300, 400), (0, 1, 2)])):
        q, k, v = inputs(rng, 500, hq, hkv, d, True)
        st = torch.tensor(cuts[0], dtype=torch.int32, device="cuda")
        out = torch.full((500, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_prefill_packed(q, k, v, st, 500, 0.1, out, ws, err)
        graphs.append((g, q, k, v, st, out, err, cuts))
    for i in range(3):
        for g, q, k, v, st, out, err, cuts in graphs:
            st.copy_(torch.tensor(cuts[i], dtype=torch.int32))
            out.fill_(7.0)
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, q, k, v, st, out, err, cuts in graphs:
            assert pa.pa_wait(err) == 0
            check(out, q, k, v, np.array(cuts[i]), 0.1)
    _, q, k, v, *_ = graphs[0]
    torch.cuda.synchronize()
    out, flag = run(pa, q, k, v, [0, 300, 500], 0.1, stream=side)
    assert flag == 0
    check(out, q, k, v, np.array([0, 300, 500]), 0.1)


@pytest.mark.gpu
def test_waits_that_run_out(pa):
    """With the bound of the in-kernel waits at a few nanoseconds the kernel gives up, sets
    the flag and returns; the same call is right again afterwards."""
    rng = np.random.default_rng(2)
    q, k, v = inputs(rng, 600, 4, 1, 128, True)
    pa.pa_set_wait_timeout_ns(1)
    try:
        _, flag = run(pa, q, k, v, [0, 600], 0.1)
    finally:
        pa.pa_set_wait_timeout_ns(0)
    assert flag & pa.PA_DEVERR_TIMEOUT
    out, flag = run(pa, q, k, v, [0, 600], 0.1)
    assert flag == 0
    check(out, q, k, v, np.array([0, 600]), 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 1, 128)])
@pytest.mark.parametrize("top", [2 ** 31 - 1, 2 ** 31 - 31, 2 ** 30, 1401])
def test_an_upper_bound_far_above_the_lengths(pa, hq, hkv, d, top):
    """max_seq_len only bounds the lengths: any larger number, up to the largest of 32 bits, gives
    the same rows, where jobs are listed and where short sequences are taken in turn."""
    rng = np.random.default_rng(hq)
    for starts in ((0, 1400), (0, 700, 701, 1300), (0, 20, 31)):
        q, k, v = inputs(rng, starts[-1], hq, hkv, d, True)
        out, flag = run(pa, q, k, v, starts, 0.1, top)
        assert flag == 0
        check(out, q, k, v, np.array(starts), 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (4, 4, 128), (8, 2, 64), (16, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_rows_between_values_that_are_not_finite(pa, hq, hkv, d, scale):
    """Infinities that a row sees and a NaN that it does not, in some dims only: its finite dims are the
    definition's, the others infinite; rows that see the NaN have it in those dims alone."""
    rng = np.random.default_rng(hq + d)
    T, at_inf, at_nan = 500, 321, 340
    q, k, v = inputs(rng, T, hq, hkv, d, False)
    v[at_inf, :, 3:5] = float("-inf")
    v[at_nan, :, 4:9] = float("nan")
    out, flag = run(pa, q, k, v, [0, T], scale)
    assert flag == 0
    clean = v.clone()
    clean[at_inf, :, 3:5], clean[at_nan, :, 4:9] = 0, 0
    ref, mass, reach = step_ops.packed_attention(*(x.double().cpu().numpy() for x in (q, k, clean)), np.array([0, T]), scale)
    bound = step_ops.attention_bound(ref, mass, reach, (0, 2.0 ** -8, 0.0))
    g = out.double().cpu().numpy()
    isinf, isnan = np.zeros(g.shape, bool), np.zeros(g.shape, bool)
    isinf[at_inf:, :, 3:5] = True
    isnan[at_nan:, :, 4:9] = True
    isinf &= ~isnan
    assert (g[isinf] == -np.inf).all() and np.isnan(g[isnan]).all()
    rest = ~isinf & ~isnan
    assert (np.abs(g - ref) <= bound)[rest].all()


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(16, 16, 64), (32, 8, 128)])
def test_rows_computed_again_take_as_long_as_they_take(pa, hq, hkv, d):
    """The last value of a prompt is not finite: the rows of its tile are computed again over thousands of
    keys, for longer than the bound of the in-kernel waits, which the CTA's other warps do not take for
    a wait that ran out; the other rows are what they are without it."""
    torch = torch_mod()
    rng = np.random.default_rng(hkv)
    T = 6144                           # whole pairs of tiles: no stream waits for a whole job of the other
    q, k, v = inputs(rng, T, hq, hkv, d, False)
    clean, flag = run(pa, q, k, v, [0, T], 0.1)
    assert flag == 0
    v[-1] = float("nan")
    pa.pa_set_wait_timeout_ns(1_000_000)
    try:
        out, flag = run(pa, q, k, v, [0, T], 0.1)
    finally:
        pa.pa_set_wait_timeout_ns(0)
    assert flag == 0
    assert torch.isnan(out[-1]).all() and torch.equal(out[:T - 256], clean[:T - 256])
    f = lambda x: x.double().cpu().numpy()
    n = 256
    for h in (0, hq - 1):
        kk, vv, qq = f(k[:, h // (hq // hkv)]), np.nan_to_num(f(v[:, h // (hq // hkv)])), f(q[T - n:T - 1, h])
        x = 0.1 * qq @ kk.T
        dead = np.arange(T)[None, :] > np.arange(T - n, T - 1)[:, None]
        x[dead] = -np.inf
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        reach = 0.1 * np.where(dead, 0.0, np.abs(qq) @ np.abs(kk).T).max(1, keepdims=True)
        bound = step_ops.attention_bound(p @ vv, p @ np.abs(vv), reach, (0, 2.0 ** -8, 0.0))
        assert (np.abs(f(out[T - n:T - 1, h]) - p @ vv) <= bound).all()
    v[:] = float("nan")
    pa.pa_set_wait_timeout_ns(1_000_000)
    try:
        out, flag = run(pa, q, k, v, [0, T], 0.1)
    finally:
        pa.pa_set_wait_timeout_ns(0)
    assert flag == 0 and torch.isnan(out).all()


@pytest.mark.gpu
def test_offsets_beyond_32_bits(pa):
    """Rows of one fused projection of more than 2^32 bytes (and an output of more), the last of 16,384
    sequences at their end, a masked value that is not finite among them."""
    torch = torch_mod()
    hq, hkv, d, S = 64, 8, 128, 16384
    rng = np.random.default_rng(14)
    n = rng.integers(0, 3, S)
    n[:8], n[-3:] = 35000, (257, 0, 140)
    starts = np.concatenate([[0], np.cumsum(n)])
    T = int(starts[-1]) + 5
    assert T * hq * d * 2 > 2 ** 32
    x = torch.zeros(T, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    from_row = int(starts[-40])
    x[from_row:] = bf16(rng.standard_normal((T - from_row, hq + 2 * hkv, d))).cuda()
    q, k, v = x.split([hq, hkv, hkv], 1)
    v[int(starts[-1]) - 1, :, 7] = float("inf")
    out, flag = run(pa, q, k, v, starts, 0.09)
    assert flag == 0 and (out[:35000:997] == 0).all()
    tail = starts[-40:] - from_row
    v[int(starts[-1]) - 1, :, 7] = 0
    got = out[from_row:].clone()
    assert torch.isinf(got[tail[-1] - 1, :, 7]).all()
    got[tail[-1] - 1] = run(pa, q, k, v, starts, 0.09)[0][int(starts[-1]) - 1]
    check(got, q[from_row:], k[from_row:], v[from_row:], tail, 0.09)
