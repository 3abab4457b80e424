"""The step plan on the GPU (block tables, slots, starts from lengths) against the
definition and against the host block manager, and the refusals."""
import ctypes as C
import os
import subprocess
import sys
import threading
import time

import numpy as np
import pytest

from oracle import step_ops
from test_abi import _gpu_visible

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def torch_mod():
    import torch
    return torch


def dev(a):
    return torch_mod().from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.skipif(_gpu_visible(), reason="passes placeholder device addresses: only where no GPU is reachable")
def test_host_validation(pa):
    L, p = pa._lib, C.c_void_p(0x10000)
    plan = lambda S=2, mb=4, fc=8, sc=4, tables=p, free=p, nf=p, slots=p, starts=p, counts=p: L.pa_step_plan(
        counts, p, S, tables, mb, free, fc, nf, slots, sc, starts, p, p, None, None)
    for bad in (dict(S=-1), dict(mb=-1), dict(fc=-1), dict(sc=-1), dict(tables=None), dict(free=None), dict(nf=None),
                dict(slots=None), dict(starts=None), dict(counts=None)):
        assert plan(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert plan(S=16385) == pa.PA_ERR_UNSUPPORTED
    assert plan(sc=(1 << 30) + 1) == pa.PA_ERR_UNSUPPORTED
    rel = lambda S=2, mb=4, fc=8, fin=p, free=p: L.pa_step_release(fin, p, S, p, mb, free, fc, p, p, p, None, None)
    for bad in (dict(S=-1), dict(mb=-1), dict(fc=-1), dict(fin=None), dict(free=None)):
        assert rel(**bad) == pa.PA_ERR_INVALID_ARG, bad
    assert rel(S=16385) == pa.PA_ERR_UNSUPPORTED


def test_tensors_on_the_host_are_refused(pa):
    torch = torch_mod()
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(AssertionError, match="CUDA device"):
        pa.pa_step_plan(z(2), z(2), z(2, 3), z(8), z(1), torch.zeros(4, dtype=torch.int64), z(3))
    with pytest.raises(AssertionError, match="seq_starts"):
        pa.pa_step_plan(z(2), z(2), z(2, 3), z(8), z(1), torch.zeros(4, dtype=torch.int64), z(2))
    with pytest.raises(AssertionError, match="CUDA device"):
        pa.pa_step_release(z(2), z(2), z(2, 3), z(8), z(1))


def case(rng, S, count_hi, ctx_hi, slack=3, pad=5, mb_extra=1):
    counts = rng.integers(0, count_hi, S, endpoint=True).astype(np.int32)
    lens = rng.integers(0, ctx_hi, S, endpoint=True).astype(np.int32)
    used = [-(-int(n) // 16) for n in lens]
    new = sum(-(-int(n + c) // 16) - u for n, c, u in zip(lens, counts, used))
    mb = max(1, max((-(-int(n + c) // 16) for n, c in zip(lens, counts)), default=1)) + mb_extra
    ids = rng.permutation(sum(used) + new + slack).astype(np.int32)
    tables = np.full((S, mb), -7, np.int32)
    at = 0
    for s, u in enumerate(used):
        tables[s, :u] = ids[at:at + u]
        at += u
    free = np.concatenate([ids[at:], np.full(at, -9, np.int32)])
    return counts, lens, tables, free, len(ids) - at, int(counts.sum()) + pad


def run_plan(pa, counts, lens, tables, free, nf, cap, inplace, offset=0):
    torch = torch_mod()
    S = len(counts)
    t = dict(counts=dev(counts), lens=dev(lens), tables=dev(tables), free=dev(free), nf=dev(np.array([nf], np.int32)))
    slots = torch.full((cap + offset,), 77, dtype=torch.int64, device="cuda")[offset:]
    starts = torch.full((S + 1,), 77, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_lens = t["lens"] if inplace else torch.full((S,), 77, dtype=torch.int32, device="cuda")
    new_nf = t["nf"] if inplace else torch.full((1,), 77, dtype=torch.int32, device="cuda")
    pa.pa_step_plan(t["counts"], t["lens"], t["tables"], t["free"], t["nf"], slots, starts, new_lens, new_nf, err)
    flag = pa.pa_wait(err)
    assert np.array_equal(t["free"].cpu().numpy(), free)          # the stack's entries are only read
    if not inplace:
        assert np.array_equal(t["lens"].cpu().numpy(), lens) and int(t["nf"]) == nf
    return (t["tables"].cpu().numpy(), slots.cpu().numpy(), starts.cpu().numpy(), new_lens.cpu().numpy(), int(new_nf)), flag


@pytest.mark.gpu
@pytest.mark.parametrize("S,count_hi,ctx_hi", [(0, 0, 0), (1, 0, 0), (1, 1, 0), (1, 1, 16), (3, 1, 40), (33, 17, 64), (256, 1, 4096),
                                               (5, 3000, 31), (64, 2048, 33), (1000, 40, 200), (1024, 1, 17), (1025, 2, 17),
                                               (5000, 3, 90), (16384, 1, 20)])
@pytest.mark.parametrize("inplace", [False, True])
def test_plan_matches_the_definition(pa, S, count_hi, ctx_hi, inplace):
    rng = np.random.default_rng(S * 31 + count_hi + ctx_hi)
    c = case(rng, S, count_hi, ctx_hi)
    ref = step_ops.step_plan(*c)
    for offset in (0, 1):     # a slot buffer that is 16-byte aligned, and one that is not
        got, flag = run_plan(pa, *c, inplace, offset)
        assert flag == 0
        for g, r, what in zip(got, ref, ("tables", "slots", "starts", "lens", "num_free")):
            assert np.array_equal(g, r), what


@pytest.mark.gpu
@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("fault", ["count", "len", "len_long", "row", "slots", "stack", "height_low", "height_high", "huge"])
def test_a_step_that_does_not_fit_changes_nothing(pa, fault, big):
    rng = np.random.default_rng(5)
    counts, lens, tables, free, nf, cap = case(rng, 200 if big else 20, 60 if big else 5, 50, slack=0, pad=3000 if big else 0)
    counts[3] = max(counts[3], 1)
    if fault == "count":
        counts[7] = -1
    elif fault == "len":
        lens[2] = -5
    elif fault == "len_long":
        lens[2] = tables.shape[1] * 16 + 1
        counts[2] = 0
    elif fault == "row":
        counts[4] = tables.shape[1] * 16 - lens[4] + 1
    elif fault == "slots":
        cap = int(counts.sum()) - 1
    elif fault == "stack":
        nf -= 1
    elif fault == "height_low":
        nf = -1
    elif fault == "height_high":
        nf = len(free) + 1
    else:
        counts[:] = 2 ** 31 - 1
    assert step_ops.step_plan(counts, lens, tables, free, nf, cap) is None
    got, flag = run_plan(pa, counts, lens, tables, free, nf, cap, False)
    assert flag == pa.PA_DEVERR_PLAN
    assert np.array_equal(got[0], tables) and (got[1] == -1).all() and (got[2] == 0).all()
    assert np.array_equal(got[3], lens) and got[4] == nf


@pytest.mark.gpu
@pytest.mark.parametrize("S,count_hi,pad", [(64, 500, 16000), (3, 9000, 9001), (5000, 8, 40001), (16384, 2, 70000)])
def test_plan_of_many_slots(pa, S, count_hi, pad):
    """Above the size at which a larger cluster shares the writing, in place and not."""
    rng = np.random.default_rng(S)
    c = case(rng, S, count_hi, 70, pad=pad)
    ref = step_ops.step_plan(*c)
    assert len(ref[1]) > 16384
    for inplace, offset in ((False, 0), (True, 1), (True, 0)):
        got, flag = run_plan(pa, *c, inplace, offset)
        assert flag == 0
        for g, r, what in zip(got, ref, ("tables", "slots", "starts", "lens", "num_free")):
            assert np.array_equal(g, r), what


@pytest.mark.gpu
def test_lengths_next_to_2_31(pa):
    """A table row of more than 2^31 tokens: lengths stop at what 32 bits hold."""
    torch = torch_mod()
    mb = 2 ** 27 + 8
    tables = torch.full((1, mb), 5, dtype=torch.int32, device="cuda")
    one = lambda *x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")
    for held, count, good in ((2 ** 31 - 1, 16, False), (2 ** 31 - 4, 4, False), (2 ** 31 - 4, 3, True)):
        lens, nf, err, slots, starts = one(held), one(3), one(0), one(*([7] * 5), dt=torch.int64), one(0, 0)
        pa.pa_step_plan(one(count), lens, tables, one(1, 2, 3), nf, slots, starts, err_flag=err)
        assert pa.pa_wait(err) == (0 if good else pa.PA_DEVERR_PLAN)
        assert int(lens) == (held + count if good else held) and int(nf) == 3
        assert slots.tolist() == ([92, 93, 94, -1, -1] if good else [-1] * 5)
        assert starts.tolist() == ([0, count] if good else [0, 0])


@pytest.mark.gpu
def test_a_negative_table_entry_is_flagged(pa):
    counts, lens = np.array([2, 1], np.int32), np.array([5, 16], np.int32)
    tables = np.array([[-1, -1], [4, -1]], np.int32)
    got, flag = run_plan(pa, counts, lens, tables, np.array([9], np.int32), 1, 3, False)
    assert flag == pa.PA_DEVERR_BLOCK_ID
    assert got[1].tolist() == [-1, -1, 9 * 16] and got[0][1].tolist() == [4, 9]


@pytest.mark.gpu
def test_a_run_of_steps_follows_the_host_manager(pa):
    """Prompts, decode steps and releases: tables, slots and the stack as the host block
    manager has them, the step captured once and replayed in place."""
    torch = torch_mod()
    rng = np.random.default_rng(11)
    S, N, mb, cap = 24, 400, 24, 1500
    order = rng.permutation(N).astype(np.int32)
    bm = pa.BlockManager(N, 16, order)
    for s in range(S):
        bm.add_seq(s)
    z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")
    counts, lens, nf, err, fin = z(S), z(S), dev(np.array([N], np.int32)), z(1), z(S)
    tables = torch.full((S, mb), -1, dtype=torch.int32, device="cuda")
    free, slots, starts = dev(order.copy()), z(cap, torch.int64), z(S + 1)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_step_plan(counts, lens, tables, free, nf, slots, starts, err_flag=err)
    for step in range(12):
        c = rng.integers(0, 60, S).astype(np.int32) if step % 5 == 0 else rng.integers(0, 2, S).astype(np.int32)
        try:
            want, pairs = bm.append_step(list(range(S)), c)
        except pa.OutOfBlocks:
            break
        assert len(pairs) == 0
        counts.copy_(dev(c))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy()[:c.sum()], want) and (slots[int(c.sum()):] == -1).all()
        if step % 3 == 2:       # some sequences end; their places take new ones
            done = rng.random(S) < 0.4
            fin.copy_(dev(done.astype(np.int32)))
            pa.pa_step_release(fin, lens, tables, free, nf, err_flag=err)
            for s in np.nonzero(done)[0]:
                bm.free(int(s))
                bm.add_seq(int(s))
        t, l = bm.build_tables(list(range(S)), mb)
        assert np.array_equal(tables.cpu().numpy(), t) and np.array_equal(lens.cpu().numpy(), l)
        h = int(nf)
        assert free[:h].tolist() == bm.free_stack() and h == bm.num_free()
    assert pa.pa_wait(err) == 0 and step >= 8


@pytest.mark.gpu
@pytest.mark.parametrize("S,mb", [(0, 4), (1, 1), (40, 9), (3000, 3), (3000, 20)])
def test_release(pa, S, mb):
    torch = torch_mod()
    rng = np.random.default_rng(S + mb)
    lens = rng.integers(0, mb * 16 + 1, S).astype(np.int32)
    done = (rng.random(S) < 0.5).astype(np.int32) * 3
    used = [-(-int(n) // 16) for n in lens]
    ids = rng.permutation(sum(used) + 4).astype(np.int32)
    tables = np.full((S, mb), -1, np.int32)
    free = np.full(len(ids), -2, np.int32)
    free[:4] = ids[:4]
    at, want_free, want_t, want_l = 4, ids[:4].tolist(), None, lens.copy()
    for s, u in enumerate(used):
        tables[s, :u] = ids[at:at + u]
        at += u
    want_t = tables.copy()
    for s in range(S):
        if done[s]:
            want_free += tables[s, :used[s]].tolist()
            want_t[s, :used[s]] = -1
            want_l[s] = 0
    td, ld, fd, nf, err = dev(tables), dev(lens), dev(free), dev(np.array([4], np.int32)), dev(np.zeros(1, np.int32))
    new_l, new_nf = torch.empty_like(ld), torch.empty_like(nf)
    pa.pa_step_release(dev(done), ld, td, fd, nf, new_l, new_nf, err)
    assert pa.pa_wait(err) == 0
    h = int(new_nf)
    assert fd[:h].tolist() == want_free and np.array_equal(td.cpu().numpy(), want_t)
    assert np.array_equal(new_l.cpu().numpy(), want_l) and int(nf) == 4 and np.array_equal(ld.cpu().numpy(), lens)
    if h > 4:   # a stack without room: nothing changes
        td, fd = dev(tables), dev(free[:h - 1])
        pa.pa_step_release(dev(done), ld, td, fd, nf, new_l, new_nf, err)
        assert pa.pa_wait(err) == pa.PA_DEVERR_PLAN
        assert np.array_equal(td.cpu().numpy(), tables) and int(new_nf) == 4
        assert np.array_equal(new_l.cpu().numpy(), lens) and np.array_equal(fd.cpu().numpy(), free[:h - 1])


def test_paged_cache_refuses_int8_without_block_scales(pa):
    from paged_kv_cache_389_b200.cache import PagedKVCache
    torch = torch_mod()
    with pytest.raises(ValueError):
        PagedKVCache(4, 2, 64, torch.int8, device="cpu")
    with pytest.raises(ValueError):
        PagedKVCache(4, 2, 64, torch.bfloat16, device="cpu", block_scales=True)


def test_binding_says_what_is_wrong(pa):
    """Arguments that are no tensors, of another rank, type or shape, or numbers out of 32 bits: an
    exception that names the argument, whatever the call."""
    torch = torch_mod()
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)
    right = dict(counts=z(2), context_lens=z(2), block_tables=z(2, 3), free_blocks=z(8), num_free=z(1),
                 slot_mapping=z(4, dt=torch.int64), seq_starts=z(3), new_context_lens=z(2), new_num_free=z(1), err_flag=z(1))
    for name, bad in (("counts", z(2, 1)), ("context_lens", z(3)), ("block_tables", z(2)), ("free_blocks", z(8, dt=torch.int64)),
                      ("num_free", z(2)), ("slot_mapping", z(4)), ("seq_starts", z(2, 2)[:, 0]), ("new_context_lens", z(1)),
                      ("new_num_free", z(1, 1)), ("err_flag", z(1, dt=torch.int64))):
        with pytest.raises(AssertionError, match=name):
            pa.pa_step_plan(**{**right, name: bad})
        with pytest.raises(TypeError, match=name):
            pa.pa_step_plan(**{**right, name: 3})
    q, k, ws = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16), z(64)
    with pytest.raises(AssertionError, match="max_seq_len"):
        pa.pa_prefill_packed(q, k, k, z(2), 2 ** 31, 0.1, q.clone(), ws)
    with pytest.raises(AssertionError, match="seq_starts"):
        pa.pa_prefill_packed(q, k, k, z(0), 4, 0.1, q.clone(), ws)
    with pytest.raises(TypeError):
        pa.pa_prefill_packed(q, k, k, z(2), 4, "0.1", q.clone(), ws)


# Kernel attributes last for the process, and one set by a larger call would hide a launch that asks for
# more shared memory than it may: a process of its own, sizes ascending, one kernel variant after the other.
AROUND_48_KB = """
import sys
import numpy as np
sys.path[:0] = ["tests", "."]
import paged_kv_cache_389_b200 as pa
import test_step_plan as t
from oracle import step_ops
for pad in (0, 4096):                      # one CTA (a few slots), a cluster
    for S in (4071, 4072, 4073, 4080, 4095, 4096, 4097):
        c = list(t.case(np.random.default_rng(S), S, 1, 20))
        c[0][:] = 0
        c[0][:1500] = 1
        c[5] = 1500 + pad
        ref = step_ops.step_plan(*c)
        got, flag = t.run_plan(pa, *c, False)
        assert flag == 0 and all(np.array_equal(g, r) for g, r in zip(got, ref)), (pad, S)
for S in (4071, 4072, 4073, 4080, 4095, 4096, 4097):
    fin, lens = np.ones(S, np.int32), np.full(S, 9, np.int32)
    tables = t.dev(np.arange(S, dtype=np.int32)[:, None])
    free, nf, err, l = t.dev(np.full(S, -5, np.int32)), t.dev(np.zeros(1, np.int32)), t.dev(np.zeros(1, np.int32)), t.dev(lens)
    pa.pa_step_release(t.dev(fin), l, tables, free, nf, err_flag=err)
    assert pa.pa_wait(err) == 0 and int(nf) == S and free.tolist() == list(range(S)), S
    assert (tables == -1).all() and (l == 0).all()
print("all sizes")
"""


@pytest.mark.gpu
def test_sizes_around_48_kb_of_shared_memory(pa):
    """12 (S + 1) bytes for the lengths and sums, and the kernel's static arrays beside them: every
    size up to and above what a launch gets without asking, in a fresh process."""
    r = subprocess.run([sys.executable, "-c", AROUND_48_KB], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all sizes" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.gpu
@pytest.mark.parametrize("S", [3, 2500])
def test_release_of_a_negative_table_entry_is_flagged(pa, S):
    """A negative id within a finished sequence's length: flagged, as the plan flags it."""
    torch = torch_mod()
    tables = np.arange(2 * S, dtype=np.int32).reshape(S, 2)
    tables[0, 1] = -4                     # inside the length
    tables[1, 1] = -4                     # behind it
    tables[2] = -4                        # of a sequence that goes on
    lens, fin = np.full(S, 20, np.int32), np.ones(S, np.int32)
    lens[1], fin[2] = 16, 0
    td, nf, err = dev(tables), dev(np.zeros(1, np.int32)), dev(np.zeros(1, np.int32))
    free, ld = torch.full((2 * S,), 77, dtype=torch.int32, device="cuda"), dev(lens)
    pa.pa_step_release(dev(fin), ld, td, free, nf, err_flag=err)
    assert pa.pa_wait(err) == pa.PA_DEVERR_BLOCK_ID
    want = [int(b) for s in range(S) if fin[s] for b in tables[s, :-(-lens[s] // 16)]]
    assert free[:int(nf)].tolist() == want and (free[int(nf):] == 77).all()
    assert ld.tolist() == [20 if s == 2 else 0 for s in range(S)]
    tables[0, 1] = 1                      # the same without it: no flag
    td, nf, ld = dev(tables), dev(np.zeros(1, np.int32)), dev(lens)
    err.zero_()
    pa.pa_step_release(dev(fin), ld, td, free, nf, err_flag=err)
    assert pa.pa_wait(err) == 0


@pytest.mark.gpu
def test_other_threads_run_while_a_call_waits(pa):
    """The launch queue holds about a thousand launches; a call behind a full one waits for room,
    and the program's other threads run meanwhile."""
    torch = torch_mod()
    counts, lens, tables, free, nf, cap = case(np.random.default_rng(0), 4, 1, 40)
    t = [dev(x) for x in (counts * 0, lens, tables, free, np.array([nf], np.int32))]
    slots, starts = torch.zeros(cap, dtype=torch.int64, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_step_plan(*t, slots, starts, err_flag=err)
    torch.cuda.synchronize()
    beats, stop = [], threading.Event()

    def beat():
        while not stop.is_set():
            beats.append(time.monotonic())
            time.sleep(0.002)

    thread = threading.Thread(target=beat)
    thread.start()
    try:
        begin = time.monotonic()
        torch.cuda._sleep(2 * 10 ** 9)             # about a second
        for _ in range(3000):
            pa.pa_step_plan(*t, slots, starts, err_flag=err)
        issued = time.monotonic()
    finally:
        stop.set()
        thread.join()
    torch.cuda.synchronize()
    assert issued - begin > 0.5, "the queue did not fill: the test says nothing"
    # a thread that waits for the interpreter gets it within milliseconds; one that cannot have it waits
    # out the sleeping kernel
    assert max(b - a for a, b in zip(beats, beats[1:])) < 0.25
    assert int(err) == 0
