"""yoco_retention against the recurrence, token by token in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

from tests import ref64


def dev32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, seed, q_lens, H, G, D, gated=True, before=None, decay=0.06, state_gain=1.0, pad=0):
        g = torch.Generator().manual_seed(seed)
        q_lens = np.asarray(q_lens)
        R, T = len(q_lens), int(q_lens.sum())
        self.qsl = np.concatenate(([0], np.cumsum(q_lens)))
        before = np.arange(R) % 2 * 5 if before is None else np.asarray(before)
        self.seq = q_lens + before
        rnd = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
        T += pad
        self.q, self.v = rnd(T, H, D).bfloat16(), rnd(T, H // G, D).bfloat16()
        self.k = (rnd(T, H // G, D) * D ** -0.5).bfloat16()
        self.decay = -decay * rnd(T, H).abs() if gated else torch.log1p(-torch.exp2(-2.0 - torch.arange(H))).float()
        n = R + 2
        self.where = np.random.default_rng(seed).permutation(n)[:R]
        self.state = rnd(n, H, D, D) * state_gain
        for r in range(R):
            if before[r] == 0:
                self.state[self.where[r]] = float("nan")  # must not be read
        self.longest, self.scale = int(q_lens.max()), D ** -0.5

    def run(self, in_place=False, stream=None, max_q=None, ws_fill=255, bits=0):
        from yoco_shared_kv_gb300 import _native as N
        T, H, D = self.q.shape
        R = len(self.seq)
        max_q = self.longest if max_q is None else max_q
        q, k, v, g, s = (x.cuda() for x in (self.q, self.k, self.v, self.decay, self.state))
        out = torch.full_like(q, 55.0)
        after = s if in_place else torch.full_like(s, 33.0)
        n = N.yoco_retention_workspace_size(R, T, max_q, H, D)
        ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda") if n else None
        err = dev32([0])
        N.yoco_retention(q, k, v, g, s, dev32(self.where), out, dev32(self.qsl), dev32(self.seq), max_q, self.scale, ws,
                         None if in_place else after, err, stream)
        torch.cuda.synchronize()
        assert int(err) == bits, hex(int(err))
        return out.cpu(), after.cpu()

    def check(self, out, after, in_place=False):
        a = [x.float().numpy() for x in (self.q, self.k, self.v, self.decay)]
        T = int(self.qsl[-1])
        g = a[3] if a[3].ndim == 1 else a[3][:T]
        state = np.nan_to_num(self.state.numpy())
        want, states = ref64.retention(a[0][:T], a[1][:T], a[2][:T], g, state, self.where, self.qsl, self.seq, self.scale)
        # the same sums of magnitudes bound every rounding: q, k, v and states by their absolute values
        mag, smag = ref64.retention(np.abs(a[0][:T]), np.abs(a[1][:T]), np.abs(a[2][:T]), g, np.abs(state), self.where,
                                    self.qsl, self.seq, abs(self.scale))
        got = out.float().numpy()
        # Outputs: half a bf16 step of the result (2^-8), of every weight and of every element of the
        # state's copy (both factors of the sum of magnitudes: 2^-8), and fp32 sums (n terms of 2^-23 each).
        # A state that only feeds later outputs of its segment holds its values in 16 bits (2^-16).
        n = T + 2 * a[0].shape[2] + 64
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -16 + n * 2.0 ** -23) * mag
        assert np.isfinite(got[:T]).all()
        worst = np.max(np.abs(got[:T] - want) / (tol + 1e-300)) if T else 0
        assert worst <= 1, worst
        assert (got[T:] == 55).all()  # rows behind the last request
        rest = np.ones(len(state), dtype=bool)
        for r in range(len(self.seq)):
            if self.qsl[r + 1] == self.qsl[r]:
                continue
            w = self.where[r]
            rest[w] = False
            # states: the fp32 sums, the factors' roundings (2^-21 each of two) and the values in 24 bits
            n = int(self.qsl[r + 1] - self.qsl[r]) + 16
            d = np.abs(after[w].numpy() - states[r]) / ((n * 2.0 ** -24 + 2.0 ** -20) * smag[r] + 1e-37)
            assert d.max() <= 1, (r, d.max())
        if not in_place:
            assert (after[torch.from_numpy(rest)] == 33).all()  # states of no request


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,gated", [(1, 1, True), (4, 2, True), (6, 3, False)])
def test_single_tokens(D, H, G, gated):
    c = Case(D + H, [1, 1, 0, 1, 1, 1], H, G, D, gated, pad=2)
    for in_place in (False, True):
        c.check(*c.run(in_place), in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,gated", [(2, 1, True), (4, 4, False)])
@pytest.mark.parametrize("lens", [[2], [64], [65, 1, 63], [0, 130, 1, 0, 3], [257, 300]])
def test_prompts(D, H, G, gated, lens):
    c = Case(len(lens) * D + H, lens, H, G, D, gated, pad=3)
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("D,H,lens", [(64, 1, [5000, 1, 700]), (128, 2, [2111, 1, 513, 900]), (256, 1, [1500, 257, 1])])
@pytest.mark.parametrize("before", [0, 7])
def test_prompts_of_several_segments(D, H, lens, before):
    c = Case(D, lens, H, 1, D, before=[before] * len(lens))
    for in_place in (False, True):
        c.check(*c.run(in_place), in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("decay", [0.0, 1e-4, 3.0, 60.0, float("inf")])
def test_decays(decay):
    """No decay at all, and decays that empty the state within a token."""
    c = Case(3, [200, 1, 77], 2, 1, 64, before=[3, 3, 0], decay=1.0)
    c.decay = torch.full_like(c.decay, -decay) if decay != 3.0 else c.decay * 3
    out, after = c.run()
    if decay == float("inf"):
        c.decay = torch.full_like(c.decay, -80.0)
    c.check(out, after)


@pytest.mark.gpu
def test_resets_between_tokens():
    """A decay of zero (log -inf) in the midst of a chunk starts anew there."""
    c = Case(4, [190], 1, 1, 128, before=[9], decay=0.01)
    for t in (0, 37, 63, 64, 150):
        c.decay[t] = float("-inf")
    out, after = c.run()
    c.decay = c.decay.clamp(min=-80)
    c.check(out, after)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G", [(64, 1), (128, 2), (256, 1)])
@pytest.mark.parametrize("at", [0, 1, 37, 64 + 63, 299, 1400])
def test_values_that_are_not_finite_stay_with_later_tokens(D, G, at):
    """Token `at` of a prompt has infinities and NaN in v, in one key or in one decay: no other
    request and no earlier token sees it."""
    lens = [70, 1500, 1, 130]
    c = Case(D + at, lens, 2, G, D, before=[0, 3, 5, 0])
    token = int(c.qsl[1]) + at
    plain, plain_state = c.run()
    x = [np.abs(y.float().numpy()) for y in (c.q, c.k, c.v)]
    mag, _ = ref64.retention(*x, c.decay.numpy(), np.nan_to_num(np.abs(c.state.numpy())), c.where, c.qsl, c.seq, c.scale)
    end, mine = int(c.qsl[2]), int(c.where[1])
    others = [int(w) for r, w in enumerate(c.where) if r != 1]
    for what in ("v", "k", "decay"):
        x = getattr(c, what)
        kept = x.clone()
        if what == "v":
            x[token, 0, 3], x[token, 0, D - 1] = float("nan"), -float("inf")
        elif what == "k":
            x[token, 0, 5] = float("nan")
        else:
            x[token, 0] = float("nan")
        out, after = c.run()
        setattr(c, what, kept)
        assert torch.equal(out[:c.qsl[1]], plain[:c.qsl[1]]) and torch.equal(out[end:], plain[end:])
        assert torch.equal(after[others], plain_state[others])
        # Tokens before: the same sums. Beside a decay that is not a number a chunk's weights are worked out
        # another way: each side rounds a weight or an element of the state's copy by 2^-8, its factor by 2^-20
        # more, and the result by 2^-8.
        a, b = out[c.qsl[1]:token].float(), plain[c.qsl[1]:token].float()
        if what != "decay":
            assert torch.equal(a, b)
        else:
            tol = 2 * (2.0 ** -8 + 2.0 ** -16) * mag[c.qsl[1]:token] + 2.0 ** -8 * (a.abs() + b.abs()).double().numpy()
            assert ((a - b).abs().numpy() <= tol).all()
        heads = slice(0, G if what != "decay" else 1)  # that read it
        bad, bad_state = out[token:end, heads], after[mine, heads]
        if what == "v":
            assert not torch.isfinite(bad[..., [3, D - 1]]).any() and not torch.isfinite(bad_state[..., [3, D - 1]]).any()
            rest = [d for d in range(D) if d not in (3, D - 1)]
            assert torch.equal(bad[..., rest], plain[token:end, heads][..., rest])
            assert torch.equal(bad_state[..., rest], plain_state[mine, heads][..., rest])
        else:
            assert torch.isnan(bad).all()
            assert torch.isnan(bad_state[:, 5] if what == "k" else bad_state).all()
        assert torch.equal(out[token:end, heads.stop:], plain[token:end, heads.stop:])


@pytest.mark.gpu
def test_a_prompt_equals_its_tokens():
    """Chunks, two calls, and single tokens walk the same recurrence (each checked against 64 bits)."""
    from yoco_shared_kv_gb300 import _native as N
    D, H, T = 128, 2, 150
    c = Case(8, [T], H, 1, D, before=[0])
    out, after = c.run()
    c.check(out, after)
    q, k, v, g = (x.cuda() for x in (c.q, c.k, c.v, c.decay))
    state = torch.full((3, H, D, D), float("nan"), device="cuda")
    where = dev32([2])
    outs = torch.zeros_like(q)
    ws = torch.empty(N.yoco_retention_workspace_size(1, T, T, H, D), dtype=torch.uint8, device="cuda")
    at = 0
    for n in (70, 1, 1, 60, 1, 17):
        s = slice(at, at + n)
        at += n
        o = torch.empty_like(q[s])
        N.yoco_retention(q[s], k[s], v[s], g[s], state, where, o, dev32([0, n]), dev32([at]), n, c.scale, ws)
        outs[s] = o
    c.check(outs.cpu(), torch.stack([state[2].cpu() if i == c.where[0] else torch.full((H, D, D), 33.0)
                                     for i in range(len(c.state))]))


@pytest.mark.gpu
def test_graph_two_streams_and_same_bits():
    from yoco_shared_kv_gb300 import _native as N
    c = Case(12, [900, 1, 300, 1], 2, 1, 128, before=[4, 4, 0, 0])
    first = c.run()
    c.check(*first)
    again = c.run(ws_fill=0)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = c.run(stream=side)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    T, H, D = c.q.shape
    q, k, v, g, s = (x.cuda() for x in (c.q, c.k, c.v, c.decay, c.state))
    out, after = torch.zeros_like(q), torch.full_like(s, 33.0)
    ws = torch.empty(N.yoco_retention_workspace_size(4, T, 900, H, D), dtype=torch.uint8, device="cuda")
    where, qsl, seq = dev32(c.where), dev32(c.qsl), dev32(c.seq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.yoco_retention(q, k, v, g, s, where, out, qsl, seq, 900, c.scale, ws, after)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out.cpu()) and torch.equal(first[1], after.cpu())


@pytest.mark.gpu
def test_bad_requests_are_left_alone():
    from yoco_shared_kv_gb300 import _native as N
    c = Case(15, [70, 1, 64, 1], 1, 1, 64, before=[2, 2, 2, 2])
    good = c.run()
    c.where[0], c.where[1] = len(c.state), -1
    out, after = c.run(bits=N.DEVERR_STATE)
    assert (out[:71] == 55).all() and torch.equal(out[71:], good[0][71:])
    c = Case(15, [70, 1, 64, 1], 1, 1, 64, before=[2, 2, 2, 2])
    c.seq[2] = 63
    out, _ = c.run(bits=N.DEVERR_POS_RANGE)
    assert (out[71:135] == 55).all() and torch.equal(out[:71], good[0][:71])
    c.seq[2] = 66
    out, _ = c.run(max_q=64, bits=N.DEVERR_OFFSETS)   # the first is longer than stated
    assert (out[:70] == 55).all() and torch.equal(out[70:], good[0][70:])
    out, _ = c.run(max_q=1, bits=N.DEVERR_OFFSETS)
    assert (out[:70] == 55).all() and torch.equal(out[70], good[0][70])
    c.qsl = np.array([0, 136, 0, 136, 136])           # running backwards, claiming tokens twice
    c.seq = np.array([138, 2, 138, 3])
    c.longest = 136
    c.run(bits=N.DEVERR_OFFSETS)


@pytest.mark.gpu
def test_states_beyond_two_gigabytes():
    """State offsets that pass 32 bits."""
    from yoco_shared_kv_gb300 import _native as N
    D, H = 256, 8
    n = (1 << 32) // (H * D * D * 4) + 1200
    c = Case(18, [3, 1, 70], H, 1, D, before=[5, 5, 5])
    state = torch.zeros(n, H, D, D, device="cuda")
    where = np.array([n - 1, n - 700, n - 1100])
    for r in range(3):
        state[where[r]] = c.state[c.where[r]].cuda()
    q, k, v, g = (x.cuda() for x in (c.q, c.k, c.v, c.decay))
    out = torch.full_like(q, 55.0)
    ws = torch.empty(N.yoco_retention_workspace_size(3, 74, 70, H, D), dtype=torch.uint8, device="cuda")
    N.yoco_retention(q, k, v, g, state, dev32(where), out, dev32(c.qsl), dev32(c.seq), 70, c.scale, ws)
    after = torch.full_like(c.state, 33.0)
    for r in range(3):
        after[c.where[r]] = state[where[r]].cpu()
    c.check(out.cpu(), after)


def test_the_reference_against_differences_of_the_parallel_form():
    """The recurrence and the closed sum agree (both in 64 bits)."""
    c = Case(1, [9, 4], 2, 2, 64, before=[3, 0])
    a = [x.float().numpy().astype(np.float64) for x in (c.q, c.k, c.v, c.decay)]
    out, _ = ref64.retention(*a, np.nan_to_num(c.state.numpy()), c.where, c.qsl, c.seq, c.scale)
    for t in (4, 8, 10):
        r = int(t >= 9)
        t0 = 9 * r
        for h in range(2):
            total = np.zeros(64)
            for j in range(t0, t + 1):
                total += np.exp(a[3][j + 1:t + 1, h].sum()) * (a[0][t, h] @ a[1][j, 0]) * a[2][j, 0]
            if r == 0:
                total += np.exp(a[3][:t + 1, h].sum()) * a[0][t, h] @ c.state[c.where[0], h].numpy().astype(np.float64)
            assert np.allclose(out[t, h], c.scale * total, rtol=1e-12, atol=1e-12)


def test_workspace_bounds():
    from yoco_shared_kv_gb300 import _native as N
    size = N.yoco_retention_workspace_size
    assert size(64, 64, 1, 8, 256) == 0
    assert size(-1, 64, 5, 8, 256) == 0 and size(4, 64, 5, 8, 96) == 0
    for D in (64, 128, 256):
        last = 0
        for T in (2, 100, 255, 256, 257, 1000, 5000, 20000, 100000, 1000001):
            n = size(10, T, T, 8, D)
            assert n >= last > -1
            last = n


def test_refusals():
    from yoco_shared_kv_gb300 import _native as N
    L, fake = N.lib, 1 << 20

    def call(q=fake, k=fake, v=fake, g=fake, s=fake, so=fake, w=fake, o=2 * fake, qsl=fake, seq=fake, R=2, T=300, mq=290,
             ns=4, H=4, Hk=2, D=128, ws=fake, ws_bytes=1 << 40, scale=1.0):
        return L.yoco_retention(q, k, v, g, 1, s, so, w, o, qsl, seq, R, T, mq, ns, H, Hk, D, ctypes.c_float(scale), ws,
                                ws_bytes, None, None)
    assert call(D=96) == N.YOCO_ERR_UNSUPPORTED
    assert call(H=5) == N.YOCO_ERR_INVALID_ARG
    assert call(H=1 << 20, Hk=1) == N.YOCO_ERR_UNSUPPORTED
    for bad in (dict(R=-1), dict(T=-1), dict(mq=0), dict(ns=0), dict(scale=float("nan")), dict(q=None), dict(k=None),
                dict(v=None), dict(g=None), dict(s=None), dict(so=None), dict(w=None), dict(o=None), dict(qsl=None),
                dict(seq=None), dict(q=fake + 2), dict(s=fake + 4), dict(ws=fake + 8), dict(q=fake, o=fake)):
        assert call(**bad) == N.YOCO_ERR_INVALID_ARG, bad
    assert call(ws=None) == N.YOCO_ERR_WORKSPACE
    assert call(ws_bytes=N.yoco_retention_workspace_size(2, 300, 290, 4, 128) - 1) == N.YOCO_ERR_WORKSPACE
    assert call(R=0, q=None) == N.YOCO_OK and call(T=0, q=None) == N.YOCO_OK
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        N.yoco_retention(z, z, z, torch.zeros(1), torch.zeros(1, 1, 64, 64), torch.zeros(1, dtype=torch.int32), z,
                         torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1, 1.0)
