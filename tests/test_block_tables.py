"""yoco_build_block_tables against a request-by-request reference (exact)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import ref64


def make(seed, R, bs, lo, hi, prefill_every=3, spare=8, max_q=None):
    """Random requests: every prefill_every-th schedules its whole prompt (or max_q of it)."""
    rng = np.random.default_rng(seed)
    seq = rng.integers(lo, hi + 1, R)
    q = np.ones(R, dtype=np.int64)
    q[::prefill_every] = seq[::prefill_every]
    if max_q:
        q = np.minimum(q, max_q)
    q[rng.random(R) < 0.1] = 0
    held, need = -(-(seq - q) // bs), -(-seq // bs)
    need = np.where(q == 0, held, need)
    width = int(-(-hi // bs)) + 2
    used, new = int(held.sum()), int((need - held).sum())
    num_blocks = used + new + spare
    perm = rng.permutation(num_blocks)
    table = np.full((R, width), -7)  # entries past the pages: left as they were
    at = 0
    for r in range(R):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    qsl = np.concatenate(([0], np.cumsum(q)))
    return dict(table=table, seq=seq, qsl=qsl, T=int(qsl[-1]), free=perm[used:], num_free=new + spare,
                num_blocks=num_blocks, bs=bs)


def run(c, pad=0, use_free=True, num_free=None, graph=False):
    from yoco_shared_kv_gb300 import _native as N
    dev = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    T = c["T"] + pad
    nf = c["num_free"] if num_free is None else num_free
    table, slots, err = dev(c["table"]), dev(np.full(T, 12345)), dev([0])
    after = dev([-5])
    args = (table, dev(c["seq"]), dev(c["qsl"]), c["num_blocks"], c["bs"], slots)
    kw = dict(free_pages=dev(c["free"]), num_free=dev([nf]), num_free_after=after) if use_free else {}
    N.yoco_build_block_tables(*args, **kw, err_word=err)
    if graph:
        torch.cuda.synchronize()
        slots.fill_(777)
        table.copy_(dev(c["table"]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            N.yoco_build_block_tables(*args, **kw, err_word=err)
        for _ in range(2):
            g.replay()
    torch.cuda.synchronize()
    want = ref64.build_block_tables(c["table"], c["seq"], c["qsl"], T, c["num_blocks"], c["bs"],
                                    c["free"] if use_free else None, nf)
    assert np.array_equal(table.cpu().numpy(), want[0])
    assert np.array_equal(slots.cpu().numpy(), want[1])
    if use_free:
        assert int(after) == want[2]
    assert int(err) == want[3], (int(err), want[3])
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("R,bs,lo,hi", [(1, 16, 1, 1), (1, 32, 33, 33), (3, 16, 1, 40), (64, 16, 15, 17),
                                        (255, 32, 1, 90), (256, 16, 1, 64), (257, 32, 31, 33),
                                        (700, 16, 1, 300), (1500, 32, 200, 201)])
def test_tables_and_slots(R, bs, lo, hi):
    for seed in range(3):
        run(make(seed, R, bs, lo, hi))


@pytest.mark.gpu
def test_one_long_prompt_and_padding():
    run(make(5, 1, 16, 20011, 20011), pad=300)
    run(make(6, 2, 32, 5000, 9000, max_q=701), pad=1)  # chunks of prompts: part of a page is held


@pytest.mark.gpu
def test_decode_only_many_requests_without_tokens():
    c = make(9, 900, 16, 1, 200, prefill_every=1000)
    c["qsl"] = np.minimum(c["qsl"], 3)  # almost every request schedules nothing
    c["T"] = 3
    run(c)


@pytest.mark.gpu
def test_free_pages_run_out():
    for short in (0, 1, 5, 40):
        c = make(11, 60, 16, 1, 200, spare=0)
        want = run(c, num_free=max(c["num_free"] - short, 0))
        assert bool(want[3] & 0x80) == (short > 0)
    c = make(11, 60, 16, 1, 200, spare=0)
    run(c, num_free=0)
    run(c, num_free=-3)                     # flagged, taken as none
    run(c, num_free=c["num_free"] + 100)    # flagged, taken as the stack's capacity


@pytest.mark.gpu
def test_bad_pages_lengths_and_offsets():
    c = make(13, 40, 16, 1, 200)
    c["free"][-2] = c["num_blocks"]         # a page outside the pool
    c["free"][-5] = -1
    run(c)
    c = make(14, 40, 16, 20, 200, prefill_every=50)
    c["table"][7, 0] = c["num_blocks"] + 3
    c["seq"][7] = 16 if c["qsl"][8] > c["qsl"][7] else c["seq"][7]
    run(c)
    c = make(15, 40, 16, 20, 200)
    c["seq"][4] = 0                          # fewer tokens than it schedules
    c["seq"][9] = 16 * c["table"].shape[1] + 1
    run(c)
    c = make(16, 10, 16, 20, 60)
    c["qsl"][3] = c["qsl"][2] - 1            # decreasing offsets: flagged, nothing written out of range
    from yoco_shared_kv_gb300 import _native as N
    dev = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    slots, err, after = dev(np.zeros(c["T"])), dev([0]), dev([0])
    N.yoco_build_block_tables(dev(c["table"]), dev(c["seq"]), dev(c["qsl"]), c["num_blocks"], 16, slots,
                              dev(c["free"]), dev([c["num_free"]]), after, err)
    assert int(err) & N.DEVERR_OFFSETS
    assert int(slots.max()) < c["num_blocks"] * 16 and int(slots.min()) >= -1


@pytest.mark.gpu
def test_without_a_stack_and_in_a_graph():
    c = make(21, 50, 16, 1, 300)
    t, _, _, _ = ref64.build_block_tables(c["table"], c["seq"], c["qsl"], c["T"], c["num_blocks"], 16, c["free"],
                                          c["num_free"])
    c["table"] = t                           # every page is there already
    run(c, use_free=False)
    run(make(22, 300, 32, 1, 100), graph=True)


@pytest.mark.gpu
def test_an_empty_stack_is_a_stack():
    """Free pages of length zero: requests that need one get none, whatever the table holds."""
    from yoco_shared_kv_gb300 import _native as N
    dev = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    table, slots, after, err = dev([[3, 4], [5, 6]]), dev([9] * 3), dev([7]), dev([0])
    N.yoco_build_block_tables(table, dev([17, 10]), dev([0, 1, 3]), 8, 16, slots, dev([]), dev([0]), after, err)
    assert slots.tolist() == [-1, 5 * 16 + 8, 5 * 16 + 9] and int(after) == 0
    assert int(err) == N.DEVERR_NO_PAGES and table.tolist() == [[3, 4], [5, 6]]


@pytest.mark.gpu
def test_empty_step():
    from yoco_shared_kv_gb300 import _native as N
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    after = z(1)
    N.yoco_build_block_tables(z(0, 4), z(0), z(1), 10, 16, z(5), z(3), z(1) + 3, after)
    assert int(after) == 3


def test_refusals():
    from yoco_shared_kv_gb300 import _native as N
    L, fake = N.lib, 1 << 20  # never dereferenced: every call below returns before a launch

    def call(bt=fake, width=4, R=2, T=3, nb=10, bs=16, free=fake, cap=5, nf=fake, after=fake + 16, slots=fake,
             qsl=fake, seq=fake):
        return L.yoco_build_block_tables(bt, width, seq, qsl, R, T, nb, bs, free, cap, nf, after, slots, None, None)
    assert call(bs=24) == N.YOCO_ERR_UNSUPPORTED
    assert call(nb=1 << 28) == N.YOCO_ERR_UNSUPPORTED       # slots would pass an int32
    assert call(T=0x7fffffff) == N.YOCO_ERR_UNSUPPORTED
    for bad in (dict(R=-1), dict(T=-1), dict(nb=0), dict(width=0), dict(cap=-1), dict(bt=None), dict(qsl=None),
                dict(seq=None), dict(slots=None), dict(nf=None), dict(after=None), dict(after=fake)):
        assert call(**bad) == N.YOCO_ERR_INVALID_ARG, bad
    assert ctypes.c_int32(N.DEVERR_NO_PAGES).value == 0x80
    with pytest.raises(ValueError):  # a CPU tensor
        z = torch.zeros(1, dtype=torch.int32)
        N.yoco_build_block_tables(z.view(1, 1), z, torch.zeros(2, dtype=torch.int32), 4, 16, z)
