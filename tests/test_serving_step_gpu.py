"""A YOCO serving step over the 4-bit cache, as an engine would run it: retention over the
step's tokens, pages taken and slots given, K/V appended, rows selected, layers attended."""
import numpy as np
import pytest
import torch

from tests import ref64
from workloads import SMALL, spec_decode

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_steps_of_a_small_engine():
    """Prompts, chunks of prompts and single tokens over five steps, the whole step captured
    in a graph of its own each time; pages and counts live on the GPU alone."""
    from yoco_shared_kv_gb300 import _native as N
    torch.manual_seed(0)
    H_q, H, D, bs, R, nb, width = 8, 2, 128, 16, 4, 40, 12
    bf = lambda *n: torch.randn(*n, device="cuda").bfloat16()  # noqa: E731
    # tokens each request schedules in each step
    plan = np.array([[40, 3, 0, 0], [20, 1, 17, 0], [1, 1, 1, 70], [1, 0, 1, 1], [2, 1, 1, 1]])
    free = i32(np.random.default_rng(1).permutation(nb))
    counts = [i32([nb]), i32([0])]
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    k, v = (torch.full((nb, H, bs, D // 2), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.full((nb, H, 2, bs, D // 32), 255, dtype=torch.uint8, device="cuda")
    state = torch.full((R + 1, H_q, D, D), float("nan"), device="cuda")
    where = i32([3, 0, 4, 1])
    err = i32([0])
    held = [[[], []] for _ in range(R)]  # every token's K and V
    rows = [[] for _ in range(R)]        # every token's retention inputs
    seq = np.zeros(R, dtype=np.int64)
    for step, q_len in enumerate(plan):
        seq = seq + q_len
        T, longest = int(q_len.sum()), int(q_len.max())
        ends = np.concatenate(([0], np.cumsum(q_len)))
        qsl, sl = i32(ends), i32(seq)
        rq, rk, rv, g = bf(T, H_q, D), bf(T, H, D) * 0.1, bf(T, H, D), -torch.rand(T, H_q, device="cuda") * 0.1
        kn, vn, q = bf(T, H, D), bf(T, H, D), bf(R, H_q, D)
        ro, out = torch.full_like(rq, 9.0), torch.full_like(q, 9.0)
        slots, rowi, cq, n = i32(np.full(T, -9)), i32(np.zeros(T)), i32(np.zeros(R + 1)), i32([0])
        rws = torch.empty(max(16, N.yoco_retention_workspace_size(R, T, longest, H_q, D)), dtype=torch.uint8, device="cuda")
        ws = torch.empty(N.yoco_cross_attn_workspace_size(R, H_q, H, D, bs, 192, N.E2M1), dtype=torch.uint8, device="cuda")

        def run():
            N.yoco_retention(rq, rk, rv, g, state, where, ro, qsl, sl, longest, D ** -0.5, rws, err_word=err)
            N.yoco_build_block_tables(table, sl, qsl, nb, bs, slots, free, counts[step % 2], counts[(step + 1) % 2], err)
            N.yoco_kv_append_e2m1(kn, vn, k, v, s, slots, err)
            N.yoco_select_cross_rows(qsl, None, rowi, cq, n, err)
            N.yoco_cross_attn_plan(table, sl, cq, 192, R, H_q, H, D, bs, nb, N.E2M1, ws, err)
            N.yoco_cross_attn_paged_e2m1(q, k, v, s, out, table, sl, cq, 192, D ** -0.5, ws, err,
                                         flags=N.YOCO_ATTN_PLANNED)
        if step % 2:
            run()
        else:  # kernels' one-time settings must not need a call before capture
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            graph.replay()
        torch.cuda.synchronize()
        assert int(err) == 0, hex(int(err))
        # what a host with all tokens at hand gets
        assert int(counts[(step + 1) % 2]) == nb - sum(-(-int(x) // bs) for x in seq)
        live = [r for r in range(R) if q_len[r]]
        assert int(n) == len(live)
        for i, r in enumerate(live):
            t = slice(int(ends[r]), int(ends[r + 1]))
            for which, new in enumerate((kn, vn)):
                held[r][which].append(new[t].float().cpu().numpy())
            rows[r].append([x[t].float().cpu().numpy() for x in (rq, rk, rv, g)])
            kv = [ref64.e2m1_values(ref64.e2m1_pack(c), b) for c, b in
                  (ref64.e2m1_encode(np.concatenate(x)) for x in held[r])]
            qq = q[i].float().cpu().numpy().astype(np.float64)
            for h in range(H_q):
                w = qq[h] @ kv[0][:, h // 4].T * D ** -0.5
                p = np.exp(w - w.max())
                p /= p.sum()
                want, mag = p @ kv[1][:, h // 4], p @ np.abs(kv[1][:, h // 4])
                # half a bf16 step of the output, half an f16 step of the weights (and as much
                # again for the fp32 sums of scores that stay below 2^5)
                assert (np.abs(out[i, h].float().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag).all()
            a = [np.concatenate([x[j] for x in rows[r]]) for j in range(4)]
            total = len(a[0])
            want, states = ref64.retention(*a, np.zeros((1, H_q, D, D)), [0], [0, total], [total], D ** -0.5)
            mag, smag = ref64.retention(*(np.abs(x) for x in a[:3]), a[3], np.zeros((1, H_q, D, D)), [0], [0, total], [total],
                                        D ** -0.5)
            m = int(q_len[r])
            tol = 2.0 ** -8 * np.abs(want[-m:]) + (2.0 ** -8 + 2.0 ** -14) * mag[-m:]
            assert (np.abs(ro[t].float().cpu().numpy() - want[-m:]) <= tol).all()
            d = np.abs(state[int(where[r])].cpu().numpy() - states[0])
            assert (d <= (total + 16) * 2.0 ** -22 * smag[0] + 1e-30).all()
        assert (out[len(live):] == 9).all()


@pytest.mark.parametrize("make", [SMALL[1], SMALL[3], SMALL[4],
                                  lambda: spec_decode(8401, num_reqs=3, ctx_lo=20, ctx_hi=300, draft=4, layers=2)])
def test_workloads_over_the_4_bit_cache(make):
    """The benchmark's workloads at small size through DeviceWorkload(kv="e2m1")."""
    import oracle
    from yoco_shared_kv_gb300 import pipeline
    wl = make()
    dw = pipeline.DeviceWorkload(wl, "cuda:0", kv="e2m1")
    dw.run_all()
    torch.cuda.synchronize()
    assert dw.error_bits() == 0
    pools = [x.cpu().numpy() for x in (dw.k_cache, dw.v_cache, dw.block_scales)]
    for ds in dw.steps:
        st = ds.step
        _, cq, _ = oracle.select_cross_rows(st.query_start_loc, st.rows_per_req)
        for layer in range(wl.layers):
            ref, tol = ref64.cross_attn_e2m1(ds.dev["q"][layer].float().cpu().numpy(), *pools, st.block_table, st.seq_lens, cq,
                                             wl.scale, int(cq[-1]))
            got = ds.out[layer].float().cpu().numpy()[: int(cq[-1])]
            assert (np.abs(got - ref) <= tol).all()
    with pytest.raises(ValueError):
        dw.fused_step(0)
