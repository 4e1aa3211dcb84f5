"""The 4-bit cache: rows bit-exact, attention against 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

from tests import ref64


def bf16(x):
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).bfloat16()


def dev32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Cache:
    """A 4-bit cache of sentinel bytes with the requests' rows encoded by the reference."""

    def __init__(self, seed, seq_lens, H, D, bs, k_gain=1.0, v_gain=1.0, spread=0, spare=3, stale=0xFF):
        rng = np.random.default_rng(seed)
        need = [-(-int(n) // bs) if n > 0 else 0 for n in seq_lens]
        self.num_blocks = sum(need) + spare
        perm = rng.permutation(self.num_blocks)
        self.table = np.full((len(need), max(max(need), 1)), -1)
        shape = (self.num_blocks, H, bs, D // 2)
        self.k, self.v = (np.full(shape, stale, dtype=np.uint8) for _ in range(2))
        self.s = np.full((self.num_blocks, H, 2, bs, D // 32), stale, dtype=np.uint8)
        at = 0
        for r, n in enumerate(seq_lens):
            pages = perm[at:at + need[r]]
            at += need[r]
            self.table[r, :need[r]] = pages
            if n <= 0:
                continue
            for pool, which, gain in ((self.k, 0, k_gain), (self.v, 1, v_gain)):
                x = rng.standard_normal((int(n), H, D)) * gain
                x *= 2.0 ** rng.integers(-spread, spread + 1, (int(n), H, D // 32)).repeat(32, -1)
                code, b = ref64.e2m1_encode(bf16(x).float().numpy())
                page, slot = pages[np.arange(n) // bs], np.arange(n) % bs
                pool[page, :, slot] = ref64.e2m1_pack(code)
                self.s[page, :, which, slot] = b
        self.bs, self.D, self.H = bs, D, H

    def on_gpu(self):
        return [torch.from_numpy(x).cuda() for x in (self.k, self.v, self.s)]


def attend(c, q, seq_lens, cqsl, scale=None, flags=0, max_rows=None, max_seq=None, planned=False, check=True, bits=0):
    from yoco_shared_kv_gb300 import _native as N
    rows, H_q, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    k, v, s = c.on_gpu()
    qd = q.cuda()
    out = torch.full_like(qd, 77.0)
    err = dev32([0])
    max_seq = max(int(max(seq_lens)), 1) if max_seq is None else max_seq
    mr = rows if max_rows is None else max_rows
    ws = torch.full((N.yoco_cross_attn_workspace_size(mr, H_q, c.H, D, c.bs, max_seq, N.E2M1),), 255,
                    dtype=torch.uint8, device="cuda")
    table, sl, cq = dev32(c.table), dev32(seq_lens), dev32(cqsl)
    if planned:
        N.yoco_cross_attn_plan(table, sl, cq, max_seq, mr, H_q, c.H, D, c.bs, c.num_blocks, N.E2M1, ws, err)
        flags |= N.YOCO_ATTN_PLANNED
    N.yoco_cross_attn_paged_e2m1(qd, k, v, s, out, table, sl, cq, max_seq, scale, ws, err, max_rows=mr, flags=flags)
    torch.cuda.synchronize()
    assert int(err) == bits, hex(int(err))
    if check:
        ref, tol = ref64.cross_attn_e2m1(q.float().numpy(), c.k, c.v, c.s, c.table, seq_lens, cqsl, scale, mr)
        got = out.float().cpu().numpy().astype(np.float64)
        n = ref.shape[0]
        worst = np.max(np.abs(got[:n] - ref) / (tol + 1e-300))
        assert np.isfinite(got[:n]).all() and worst <= 1.0, worst
        assert (got[n:] == 77.0).all()  # rows behind the last request stay
    return out


def queries(seed, rows, H_q, D, gain=1.0):
    return bf16(np.random.default_rng(seed + 1000).standard_normal((rows, H_q, D)) * gain)


# ------------------------------------------------------------------- rows

@pytest.mark.gpu
@pytest.mark.parametrize("T,H,D,bs", [(1, 1, 128, 16), (3, 2, 256, 16), (130, 3, 128, 32), (77, 5, 256, 32),
                                      (2500, 1, 128, 16)])
def test_append_and_gather_are_exact(T, H, D, bs):
    from yoco_shared_kv_gb300 import _native as N
    rng = np.random.default_rng(T)
    num_blocks = T // bs + 5
    slots = rng.permutation(num_blocks * bs)[:T]
    x = [bf16(rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-40, 40, (T, H, D // 32)).repeat(32, -1))
         for _ in range(2)]
    # ties, halves of the smallest code, the block's limit, zeros of both signs
    x[0][0, 0, :32] = bf16([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5,
                            0, -0.0, .2490234375, .251953125, 4.96875, 5.03125, 1, 2, 3, 4, .5, 1.5, -.5, -1.5, -3, -4])
    shape = (num_blocks, H, bs, D // 2)
    k, v = (torch.full(shape, 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.full((num_blocks, H, 2, bs, D // 32), 0xEE, dtype=torch.uint8, device="cuda")
    err = dev32([0])
    sl = dev32(slots)
    N.yoco_kv_append_e2m1(x[0].cuda(), x[1].cuda(), k, v, s, sl, err)
    out = [torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    N.yoco_kv_gather_e2m1(k, v, s, sl, *out, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    page, at = slots // bs, slots % bs
    for which, (pool, o) in enumerate(((k, out[0]), (v, out[1]))):
        code, b = ref64.e2m1_encode(x[which].float().numpy())
        want = np.full(shape, 0xEE, dtype=np.uint8)
        want[page, :, at] = ref64.e2m1_pack(code)
        assert np.array_equal(pool.cpu().numpy(), want)
        want = np.full((num_blocks, H, bs, D // 32), 0xEE, dtype=np.uint8)
        want[page, :, at] = b
        assert np.array_equal(s[:, :, which].cpu().numpy(), want)
        assert np.array_equal(o.float().cpu().numpy(), ref64.e2m1_values(ref64.e2m1_pack(code), b))


@pytest.mark.gpu
def test_append_of_extremes():
    from yoco_shared_kv_gb300 import _native as N
    x = torch.zeros(6, 1, 128, dtype=torch.bfloat16)
    x[0, 0, 3] = float("inf")
    x[0, 0, 40] = float("-inf")
    x[1, 0, 5] = float("nan")
    x[2] = torch.finfo(torch.bfloat16).max
    x[3] = 2.0 ** -130                      # a subnormal bf16
    x[4, 0, :] = bf16(np.linspace(-3e-39, 3e-39, 128))
    x[5, 0, 0] = -torch.finfo(torch.bfloat16).max
    k, v = (torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.zeros(1, 1, 2, 16, 4, dtype=torch.uint8, device="cuda")
    o = [torch.empty(6, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sl = dev32(np.arange(6))
    N.yoco_kv_append_e2m1(x.cuda(), (-x).cuda(), k, v, s, sl)
    N.yoco_kv_gather_e2m1(k, v, s, sl, *o)
    for sign, got, pool, which in ((1, o[0], k, 0), (-1, o[1], v, 1)):
        code, b = ref64.e2m1_encode((sign * x).float().numpy())
        assert np.array_equal(s[0, 0, which, :6].cpu().numpy(), b[:, 0])
        assert np.array_equal(pool[0, 0, :6].cpu().numpy(), ref64.e2m1_pack(code)[:, 0])
        assert torch.isfinite(got).all()


@pytest.mark.gpu
def test_rows_skip_padding_and_bad_slots():
    from yoco_shared_kv_gb300 import _native as N
    T, H, D, bs, nb = 40, 2, 128, 16, 4
    x = torch.randn(T, H, D, device="cuda").bfloat16()
    slots = np.full(T, -1)
    slots[3], slots[9] = 17, nb * bs  # one row, one past the pool
    k, v = (torch.full((nb, H, bs, D // 2), 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.full((nb, H, 2, bs, D // 32), 1, dtype=torch.uint8, device="cuda")
    err = dev32([0])
    N.yoco_kv_append_e2m1(x, x, k, v, s, dev32(slots), err)
    assert int(err) == N.DEVERR_PAGE_RANGE
    changed = (k != 1).any(-1).any(1).nonzero().tolist()
    assert changed == [[1, 1]]
    out = [torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    err.zero_()
    N.yoco_kv_gather_e2m1(k, v, s, dev32(slots), *out, err)
    assert int(err) == N.DEVERR_PAGE_RANGE
    for o in out:
        assert o[3].abs().sum() > 0 and o.abs().sum() == o[3].abs().sum()
    dup = dev32([17] * T)  # the same slot read many times
    N.yoco_kv_gather_e2m1(k, v, s, dup, *out, err)
    assert (out[0] == out[0][:1]).all()


# -------------------------------------------------------------- attention

SHAPES = [(8, 2, 256, 16), (16, 1, 128, 32), (8, 2, 128, 32), (1, 1, 128, 16), (3, 1, 256, 32), (24, 2, 128, 16),
          (16, 1, 256, 16), (12, 1, 256, 32), (16, 2, 128, 16), (5, 5, 128, 32), (9, 1, 128, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("H_q,H,D,bs", SHAPES)
def test_attention_one_row_each(H_q, H, D, bs):
    seq = [1, bs - 1, bs, bs + 1, 2, 700, 3 * bs, 5, 1201]
    c = Cache(H_q * D + bs, seq, H, D, bs)
    q = queries(H_q, len(seq), H_q, D)
    cq = np.arange(len(seq) + 1)
    a = attend(c, q, seq, cq)
    b = attend(c, q, seq, cq, planned=True)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    attend(c, q, seq, cq, flags=0x1 | 0x4)   # backwards, with the cache hints


@pytest.mark.gpu
@pytest.mark.parametrize("H_q,H,D,bs", SHAPES)
@pytest.mark.parametrize("rows", [2, 4, 7])
def test_attention_several_rows(H_q, H, D, bs, rows):
    seq = [rows, bs + 1, 333, 5 * bs + rows - 1, rows + 1]
    c = Cache(rows * D + H_q, seq, H, D, bs)
    q = queries(H_q + rows, rows * len(seq), H_q, D)
    cq = np.arange(len(seq) + 1) * rows
    attend(c, q, seq, cq)
    attend(c, q, seq, cq, flags=0x1)


@pytest.mark.gpu
@pytest.mark.parametrize("D,bs,H_q,H", [(256, 16, 8, 2), (128, 32, 16, 1), (128, 16, 4, 1)])
def test_attention_long(D, bs, H_q, H):
    seq = [20011, 1, 9000]
    c = Cache(3, seq, H, D, bs)
    attend(c, queries(3, 3, H_q, D), seq, np.arange(4))


@pytest.mark.gpu
@pytest.mark.parametrize("D,bs", [(128, 16), (256, 32)])
def test_attention_ragged_batches(D, bs):
    """Requests without rows, rows without keys, and rows behind the last request."""
    seq = [40, 0, 2, 100, 7]
    cq = np.array([0, 2, 2, 5, 5, 6])        # the third request has 3 rows of 2 keys
    c = Cache(5, seq, 1, D, bs)
    for flags in (0, 1):
        out = attend(c, queries(5, 9, 4, D), seq, cq, bits=0x4, flags=flags)
        assert (out[2] == 0).all()
    attend(c, queries(5, 9, 4, D), seq, cq, bits=0x4, max_rows=3)  # later rows are not looked at


@pytest.mark.gpu
@pytest.mark.parametrize("D,bs,H_q", [(128, 16, 4), (256, 16, 8), (128, 32, 16)])
def test_attention_of_wide_ranges(D, bs, H_q):
    """Scales of a row up to 2^12 apart, huge and tiny queries, steep scores."""
    seq = [1, 50, 333]
    c = Cache(7, seq, 1, D, bs, spread=3)
    for gain, scale in ((2.0 ** 40, 2.0 ** -42), (2.0 ** -60, 2.0 ** 58), (1.0, 1.0)):
        attend(c, queries(8, 3, H_q, D, gain), seq, np.arange(4), scale=scale)
    for kg, vg in ((2.0 ** -30, 2.0 ** 60), (2.0 ** 20, 2.0 ** -50)):
        c = Cache(9, seq, 1, D, bs, k_gain=kg, v_gain=vg)
        attend(c, queries(9, 3, H_q, D), seq, np.arange(4), scale=1.0 / (16 * kg))
    q = queries(10, 3, H_q, D)
    q[:, :, :2] = 0
    q[1] = 0                                   # a row of zeros: the mean of V
    attend(c, q, seq, np.arange(4), scale=1e-7)
    attend(c, queries(10, 3, H_q, D, 2.0 ** -100), seq, np.arange(4), scale=1e-30)  # scores vanish: the mean again


@pytest.mark.gpu
def test_attention_bad_pages_and_lengths():
    seq = [100, 60, 40]
    c = Cache(11, seq, 1, 128, 16)
    q = queries(11, 3, 4, 128)
    c.table[1, 1] = c.num_blocks
    attend(c, q, seq, np.arange(4), bits=0x1, check=False)
    c.table[1, 1] = -1
    attend(c, q, seq, np.arange(4), bits=0x1, check=False)
    c = Cache(11, seq, 1, 128, 16)
    attend(c, q, [100, 60, 40], np.arange(4), bits=0x2, max_seq=50)  # flagged, all keys attended
    attend(c, q, [10 ** 6, 60, 40], np.arange(4), bits=0x2, check=False, max_seq=10 ** 6)


@pytest.mark.gpu
def test_stale_bytes_do_not_matter():
    seq = [37, 5, 65]
    q = queries(12, 3, 8, 256)
    outs = [attend(Cache(12, seq, 2, 256, 16, stale=b), q, seq, np.arange(4)) for b in (0xFF, 0x00, 0x7F)]
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


@pytest.mark.gpu
def test_layers_in_a_graph_and_on_two_streams():
    from yoco_shared_kv_gb300 import _native as N
    seq, H_q, H, D, bs = [700, 33, 1500, 16], 8, 2, 256, 16
    c = Cache(13, seq, H, D, bs)
    k, v, s = c.on_gpu()
    q = torch.stack([queries(20 + i, 4, H_q, D) for i in range(3)]).cuda()
    table, sl, cq = dev32(c.table), dev32(seq), dev32(np.arange(5))
    size = N.yoco_cross_attn_workspace_size(4, H_q, H, D, bs, 1500, N.E2M1)
    err = dev32([0])

    def step(ws, out, stream=None):
        N.yoco_cross_attn_plan(table, sl, cq, 1500, 4, H_q, H, D, bs, c.num_blocks, N.E2M1, ws, err, stream)
        for i in range(3):
            N.yoco_cross_attn_paged_e2m1(q[i], k, v, s, out[i], table, sl, cq, 1500, D ** -0.5, ws, err, stream,
                                         flags=N.YOCO_ATTN_PLANNED | (N.YOCO_ATTN_REVERSE if i % 2 else 0)
                                         | (N.YOCO_ATTN_OVERLAP if i else 0))
    ws = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    outs = [torch.zeros_like(q) for _ in range(3)]
    step(ws[0], outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(ws[1], outs[1])
    for _ in range(3):
        outs[1].zero_()
        g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(ws[2], outs[2], side)
    torch.cuda.synchronize()
    assert int(err) == 0
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    for i in range(3):
        ref, tol = ref64.cross_attn_e2m1(q[i].float().cpu().numpy(), c.k, c.v, c.s, c.table, seq, np.arange(5),
                                         D ** -0.5, 4)
        assert (np.abs(outs[0][i].float().cpu().numpy() - ref) <= tol).all()


@pytest.mark.gpu
def test_pages_beyond_two_gigabytes():
    """Offsets into the pools that pass 32 bits (codes of 2.1 GiB a pool)."""
    from yoco_shared_kv_gb300 import _native as N
    H, D, bs = 4, 256, 32
    nb = (1 << 31) // (H * bs * D // 2) + 40
    k, v = (torch.zeros(nb, H, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.ones(nb, H, 2, bs, D // 32, dtype=torch.uint8, device="cuda")
    seq = [70, 33]
    pages = np.array([[nb - 1, nb - 20, nb - 3], [nb - 7, 2, 0]])
    rng = np.random.default_rng(5)
    new = [bf16(rng.standard_normal((sum(seq), H, D))) for _ in range(2)]
    slots = np.concatenate([pages[r][np.arange(n) // bs] * bs + np.arange(n) % bs for r, n in enumerate(seq)])
    err = dev32([0])
    N.yoco_kv_append_e2m1(new[0].cuda(), new[1].cuda(), k, v, s, dev32(slots), err)
    q = queries(4, 2, 8, D)
    out = torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(N.yoco_cross_attn_workspace_size(2, 8, H, D, bs, 70, N.E2M1), dtype=torch.uint8, device="cuda")
    N.yoco_cross_attn_paged_e2m1(q.cuda(), k, v, s, out, dev32(pages), dev32(seq), dev32([0, 1, 2]), 70, D ** -0.5, ws,
                                 err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kk, vv = (torch.zeros(6, H, bs, D // 2, dtype=torch.uint8) for _ in range(2))
    ss = torch.ones(6, H, 2, bs, D // 32, dtype=torch.uint8)
    for i, p in enumerate(pages.reshape(-1)):
        kk[i], vv[i], ss[i] = k[p].cpu(), v[p].cpu(), s[p].cpu()
    ref, tol = ref64.cross_attn_e2m1(q.float().numpy(), kk.numpy(), vv.numpy(), ss.numpy(), np.arange(6).reshape(2, 3),
                                     seq, [0, 1, 2], D ** -0.5, 2)
    assert (np.abs(out.float().cpu().numpy() - ref) <= tol).all()
    code, b = ref64.e2m1_encode(new[0].float().numpy())
    assert np.array_equal(k[slots // bs, :, slots % bs].cpu().numpy(), ref64.e2m1_pack(code))


# ------------------------------------------------------------ on the host

def test_the_format_by_hand():
    code, b = ref64.e2m1_encode(np.array([[6.0] + [0.25, 0.75, 5.0, -1.25, 1.75] + [0.0] * 26]))
    assert b[0, 0] == 127 and code[0, :6].tolist() == [7, 0, 2, 6, 10, 4]
    assert ref64.e2m1_encode(np.full((1, 32), 6.0078125))[1][0, 0] == 128
    assert ref64.e2m1_encode(np.zeros((1, 32)))[1][0, 0] == 1
    assert ref64.e2m1_encode(np.full((1, 32), 3e38))[1][0, 0] == 251
    x = np.random.default_rng(0).standard_normal((50, 64))
    code, b = ref64.e2m1_encode(x)
    back = ref64.e2m1_values(ref64.e2m1_pack(code), b)
    unit = np.ldexp(1.0, b.astype(int) - 127).repeat(32, -1)
    assert (np.abs(back - x) <= np.maximum(0.25 * unit, np.abs(x) / 5 + 1e-9)).all()


def test_refusals_of_rows():
    from yoco_shared_kv_gb300 import _native as N
    L, fake = N.lib, 1 << 20

    def call(fn, a=fake, b=fake, c=fake, d=fake, e=fake, f=fake, T=3, nb=10, bs=16, H=2, D=128):
        return getattr(L, fn)(a, b, c, d, e, f, T, nb, bs, H, D, None, None)
    for fn in ("yoco_kv_append_e2m1", "yoco_kv_gather_e2m1"):
        assert call(fn, D=64) == N.YOCO_ERR_UNSUPPORTED
        assert call(fn, bs=8) == N.YOCO_ERR_UNSUPPORTED
        assert call(fn, nb=1 << 28) == N.YOCO_ERR_UNSUPPORTED
        for bad in (dict(T=-1), dict(nb=0), dict(H=0), dict(a=None), dict(b=None), dict(c=None), dict(d=None),
                    dict(e=None), dict(f=None), dict(a=fake + 8)):
            assert call(fn, **bad) == N.YOCO_ERR_INVALID_ARG, (fn, bad)
        assert call(fn, T=0, a=None) == N.YOCO_OK
    with pytest.raises(ValueError):
        z = torch.zeros(1, 1, 16, 64, dtype=torch.uint8)
        N.yoco_kv_append_e2m1(torch.zeros(1, 1, 128, dtype=torch.bfloat16), torch.zeros(1, 1, 128, dtype=torch.bfloat16),
                              z, z, torch.zeros(1, 1, 2, 16, 4, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32))


def test_refusals_of_attention():
    from yoco_shared_kv_gb300 import _native as N
    L, fake = N.lib, 1 << 20

    def attn(D=128, bs=16, H_q=8, H=2, flags=0, ws=fake, ws_bytes=None, sc=fake, k=fake, R=2, rows=2, scale=0.1, nb=100):
        need = N.yoco_cross_attn_workspace_size(2, H_q, H, D, bs, 64, N.E2M1)
        return L.yoco_cross_attn_paged_e2m1(fake, k, fake, sc, fake, fake, 4, fake, fake, R, rows, 64, H_q, H, D, bs, nb,
                                            ctypes.c_float(scale), flags, ws, need if ws_bytes is None else ws_bytes, None,
                                            None)
    assert attn(D=64) == N.YOCO_ERR_UNSUPPORTED
    assert attn(bs=64) == N.YOCO_ERR_UNSUPPORTED
    assert attn(H_q=34) == N.YOCO_ERR_UNSUPPORTED
    assert attn(H_q=9) == N.YOCO_ERR_INVALID_ARG
    assert attn(flags=0x10) == N.YOCO_ERR_INVALID_ARG
    assert attn(sc=None) == N.YOCO_ERR_INVALID_ARG
    assert attn(sc=fake + 4) == N.YOCO_ERR_INVALID_ARG
    assert attn(k=None) == N.YOCO_ERR_INVALID_ARG
    assert attn(scale=float("nan")) == N.YOCO_ERR_INVALID_ARG
    assert attn(ws=None) == N.YOCO_ERR_WORKSPACE
    assert attn(ws_bytes=100) == N.YOCO_ERR_WORKSPACE
    assert attn(nb=1 << 28) == N.YOCO_ERR_UNSUPPORTED
    assert attn(R=0) == N.YOCO_OK and attn(rows=0) == N.YOCO_OK
    # the cache has entries of its own: the others refuse its dtype
    assert L.yoco_cross_attn_paged(fake, fake, fake, fake, fake, 4, fake, fake, 2, 2, 64, 8, 2, 128, 16, 100,
                                   ctypes.c_float(0.1), N.YOCO_E2M1, 0, fake, 1 << 30, None, None) == N.YOCO_ERR_UNSUPPORTED
    assert L.yoco_kv_append(fake, fake, fake, fake, fake, 4, fake, fake, 1, 1, 10, 16, 2, 128, N.YOCO_E2M1, None,
                            None) == N.YOCO_ERR_UNSUPPORTED
    assert L.yoco_cross_decode_step(fake, fake, fake, fake, fake, fake, fake, fake, 4, fake, fake, 2, 64, 8, 2, 128, 16,
                                    100, ctypes.c_float(0.1), N.YOCO_E2M1, 0, fake, 1 << 30, None,
                                    None) == N.YOCO_ERR_UNSUPPORTED
    assert L.yoco_cross_attn_paged_noalloc(fake, fake, fake, fake, fake, 4, fake, fake, 2, 2, 64, 8, 2, 128, 16, 100,
                                           ctypes.c_float(0.1), N.YOCO_E2M1, None, None) == N.YOCO_ERR_UNSUPPORTED


def test_traffic_of_the_4_bit_cache():
    from yoco_shared_kv_gb300 import _native as N
    total, per = N.yoco_cross_decoder_bytes([0, 1, 5, 5], None, [33, 40, 9], 3, 8, 2, 256, 16, N.E2M1)
    page = 4 + 2 * 16 * 8
    want = [3 * (n * 2 * 256 + 2 * 8 * 256 * 2 + page * -(-n // 16) * 2) for n in (33, 40)] + [0]
    assert per.tolist() == want and total == sum(want)


def test_workspace_does_not_grow_with_the_context():
    from yoco_shared_kv_gb300 import _native as N
    for D in (128, 256):
        for bs in (16, 32):
            for G in (1, 4, 8, 16):
                n = N.yoco_cross_attn_workspace_size(64, 2 * G, 2, D, bs, 1 << 20, N.E2M1)
                assert n > 0 and n == N.yoco_cross_attn_workspace_size(4096, 2 * G, 2, D, bs, 512, N.E2M1)
    assert N.yoco_cross_attn_workspace_size(64, 8, 2, 64, 16, 512, N.E2M1) == 0
