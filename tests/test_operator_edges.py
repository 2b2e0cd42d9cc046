"""Edges of the operators beside the GEMV: what a caller can hand them that the
plain cases of test_operators.py do not, against the same 64-bit forms. GPU
tests need a B200."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_gemv_stagq_b200 as Q
from tests import operator_oracle as R
from tests.test_operators import BF16, EFORMAT, EINVAL, F16, F32, Case, assert_rounded, rnd

gpu = pytest.mark.gpu


# ------------------------------------------------------------------- masses

@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens", [2, 40, 700])
def test_a_query_that_is_not_finite_spoils_no_mass_that_it_does_not_see(tokens, bad):
    # the oldest of three new tokens, one of KV head 0's two query heads: it
    # does not see the last two positions, whose masses come from the others
    c = Case([tokens, 5], 2, 128, 16, 64, F16)
    q = rnd((6, 4 * 128), 3, F16)
    q[0, 128 + 7] = bad
    mass = torch.zeros(2, 2, c.width * 16, device="cuda")
    out = c.attend(q.cuda(), 3, mass).view(2, 3, 4, 128).cpu()
    clean = q.clone()
    clean[0, 128 + 7] = 0
    want, p, bound, p_bound = R.attention(clean.view(2, 3, 4, 128), c.k, c.v, c.lens_l, 3, 128 ** -0.5)
    seen = max(tokens - 2, 0)
    if seen:
        assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(mass[0, 0, :seen]).all()
    else:
        assert not out[0, 0, 1].any()
    others = torch.ones(2, 3, 4, dtype=torch.bool)
    others[0, 0, 1] = False
    assert_rounded(out[others], want[others], F16, bound[others][:, None])
    got = mass.double().cpu()
    for b, h, lo in ((0, 0, seen), (0, 1, 0), (1, 0, 0), (1, 1, 0)):
        n = c.lens_l[b]
        assert ((got[b, h, lo:n] - p[b, h, lo:n]).abs() <= p_bound[b, h, lo:n] + 2.0 ** -24 * p[b, h, lo:n]).all(), (b, h)
        assert not got[b, h, n:].any()
    Q.stagq_ops_check(0)


# ----------------------------------------------------------------- eviction

@gpu
@pytest.mark.parametrize("dim,group,budget", [(64, 32, 40), (128, 128, 24)])
def test_evict_of_a_token_on_a_bad_page_leaves_zeros_and_not_the_fresh_pages_bytes(dim, group, budget):
    heads, page, n = 2, 16, 40
    c = Case([n, 33], heads, dim, page, group, F16, spare=6)  # what no call wrote is 0xFF: NaN pairs
    fresh = c.unused.reshape(2, 3).cuda()
    mass = torch.rand(2, heads, c.width * page, generator=torch.Generator().manual_seed(1))
    mass[0, :, 16:32] += 1  # the bad page's tokens are kept
    table = c.table.clone()
    kept, new_lens = torch.empty(2, heads, budget, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    new_mass = torch.empty(2, heads, budget, device="cuda")
    k, v = (torch.empty(2 * budget, heads * dim, device="cuda") for _ in range(2))
    for number in (-1, c.pool.shape[0]):
        c.pool[c.unused.long().cuda()] = 0xFF
        table[0, 1] = number
        Q.stagq_kv_evict(c.cache, table, c.lens, mass.cuda(), fresh, budget, 3, kept, new_lens, new_mass)
        with pytest.raises(Q.StagqError) as e:
            Q.stagq_ops_check(0)
        assert e.value.status == EFORMAT
        Q.stagq_kv_read(c.cache, fresh, new_lens, k, v, budget)
        Q.stagq_ops_check(0)
        for b, m in enumerate((n, 33)):
            for h in range(heads):
                want = R.keep(mass[b, h].numpy(), m, budget, 3)
                assert kept[b, h].tolist() == want + [-1] * (budget - len(want))
                assert torch.equal(new_mass[b, h, :len(want)].cpu(), mass[b, h, want])
                for got, values in ((k, c.k), (v, c.v)):
                    x = values[b, want, h].clone()
                    if b == 0:
                        x[[i for i, t in enumerate(want) if 16 <= t < 32]] = 0
                    assert_rounded(got.view(2, budget, heads, dim)[b, :len(want), h], x, F32)


def _evict_in_c(**kw):
    """stagq_kv_evict of 2 sequences on pointers that are never read, as every call here is refused."""
    f = dict(heads=2, page=16, table=8192, fresh=16384, batch=2, width=4, lens=1, max_len=64, mass=2, mb=128, mh=64, budget=8,
             recent=2, kept=3, new_lens=4, new_mass=5, nb=128, nh=64, cap=64)
    f.update(kw)
    cache = Q._KvCache(4096, 4, f["heads"], 128, f["page"], 128, 0, 0)
    t, fresh = (Q._KvTable(f[n], f["width"], f["batch"], f["width"]) for n in ("table", "fresh"))
    p = {n: ctypes.c_void_p(4096 * f[n]) for n in ("lens", "mass", "kept", "new_lens", "new_mass")}
    r = ctypes.byref
    return Q.lib().stagq_kv_evict(r(cache), r(t), p["lens"], f["max_len"], p["mass"], f["mb"], f["mh"], f["budget"], f["recent"],
                                  r(fresh), p["kept"], p["new_lens"], p["new_mass"], f["nb"], f["nh"], f["cap"], None)


@pytest.mark.parametrize("kw", [dict(new_lens=1), dict(new_mass=2), dict(fresh=8192)])
def test_evict_refuses_to_work_in_place(kw):
    assert _evict_in_c(**kw) == EINVAL
    assert "must not be" in Q.lib().stagq_last_error().decode()


@pytest.mark.parametrize("kw", [dict(lens=0), dict(mass=0), dict(kept=0), dict(new_lens=0), dict(new_mass=0), dict(fresh=0), dict(table=0),
                                dict(max_len=0), dict(max_len=65), dict(budget=0), dict(budget=65), dict(recent=-1), dict(recent=9),
                                dict(cap=7), dict(mh=63), dict(nh=63), dict(mb=127), dict(nb=127), dict(page=8), dict(batch=0)])
def test_evict_refuses_what_does_not_fit(kw):
    assert _evict_in_c(**kw) == EINVAL
    assert "must not be" not in Q.lib().stagq_last_error().decode()  # for its own reason


@pytest.mark.parametrize("kw", [dict(heads=1, batch=1, cap=2 ** 31 - 1, nh=2 ** 31, nb=2 ** 31),  # the kernel rounds new_cap up
                                dict(heads=1, batch=1, cap=2 ** 30 + 1, nh=2 ** 31, nb=2 ** 31),
                                # heads times chunks of new_cap is 2^67 and wraps to a negative number
                                dict(heads=4096, batch=2 ** 31 - 1, cap=2 ** 30, nh=2 ** 30, nb=2 ** 42, mb=2 ** 18)])
def test_evict_refuses_sizes_that_its_indices_do_not_hold(kw):
    assert _evict_in_c(**kw) == EINVAL


# ------------------------------------------------------------ waits that run out

ETIMEOUT = 7


def gave_up():
    with pytest.raises(Q.StagqError) as e:
        Q.stagq_ops_check(0)
    Q.stagq_ops_check(0)  # reported once
    return e.value.status == ETIMEOUT


# tiles of 16, 32 and 64 tokens (K shared by clusters, and not), pairs on 128 and on 256 channels; few K blocks, and
# many times the ring's
STALLED = [(1, 4096, 300), (20, 512, 1000), (64, 32768, 640), (64, 256, 40000), (129, 640, 384), (1100, 2048, 1500), (2049, 4096, 2600)]


@gpu
@pytest.mark.parametrize("n,inp,out", STALLED)
def test_gemm_i8_ends_when_a_wait_runs_out_and_works_again(n, inp, out):
    g = torch.Generator(device="cuda").manual_seed(n)
    a, b = (torch.randint(-127, 128, (r, inp), generator=g, device="cuda", dtype=torch.int8) for r in (n, out))
    xs, ws = torch.ones(n, device="cuda"), torch.full((out,), 2.0 ** -10, device="cuda")
    y = torch.empty(n, out, device="cuda")
    for stall in (2000, 50000):
        Q.stagq_debug_stall_ops(0, stall)
        try:
            Q.stagq_gemm_i8(a, xs, b, ws, inp, y)
        finally:
            Q.stagq_debug_stall_ops(0, 0)
        assert gave_up()
        y.fill_(float("nan"))
        Q.stagq_gemm_i8(a, xs, b, ws, inp, y)
        Q.stagq_ops_check(0)
        assert torch.equal(y, (a.double() @ b.double().T).float() * 2.0 ** -10)  # |sum| < 2^29: one rounding on both sides


@gpu
@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("lens,heads,group,n_new", [([1], 1, 128, 1), ([777], 2, 128, 1), ([900, 0, 4000], 2, 32, 1), ([700, 33], 2, 64, 4)])
def test_attention_ends_when_a_wait_runs_out_and_works_again(lens, heads, group, n_new, tracked):
    c = Case(lens, heads, 128, 16, group, F16)
    q = rnd((len(lens) * n_new, heads * 4 * 128), 5, F16).cuda()
    for stall in (2000, 50000):
        Q.stagq_debug_stall_ops(0, stall)
        try:
            c.attend(q, n_new, torch.zeros(len(lens), heads, c.width * 16, device="cuda") if tracked else None)
        finally:
            Q.stagq_debug_stall_ops(0, 0)
        assert gave_up()
        c.check(heads * 4, n_new, q=q.cpu(), tracked=tracked)


def test_stall_hook_refuses_bad_devices():
    assert Q.lib().stagq_debug_stall_ops(-1, 0) == EINVAL and Q.lib().stagq_debug_stall_ops(64, 0) == EINVAL


# ----------------------------------------- what an earlier kernel of the stream writes

def test_kernels_read_inputs_of_earlier_kernels_with_plain_loads():
    """The operators are launched before the kernel ahead of them in the stream
    has ended (programmatic dependent launch), so data that it writes changes
    within their lifetime: the read-only path, which must not see such data, is
    not for them."""
    import os
    csrc = os.path.join(os.path.dirname(Q.__file__), "csrc")
    for name in ("gemm_i8.cu", "kv_cache.cu", "kv_attention.cu", "ops_common.cuh"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert "ld.global.nc" not in text and "__ldg" not in text, name


@gpu
@pytest.mark.parametrize("n", [3, 40, 300])
def test_buffers_used_again_by_the_next_call(n):
    # a layer after another through the same xq, xscale and page table, each step written by the kernel before it
    inp, out, layers = 1024, 900, 12
    g = torch.Generator().manual_seed(n)
    xs = [(torch.randn(n, inp, generator=g) * 2.0 ** (i % 5)).to(F16).cuda() for i in range(layers)]
    w = torch.randint(-127, 128, (out, inp), generator=g, dtype=torch.int8).cuda()
    ws = torch.rand(out, generator=g).cuda() * 0.01
    xq, xscale = torch.empty(n, inp, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    want, got = [], [torch.empty(n, out, device="cuda") for _ in xs]
    for x in xs:
        q, s, y = torch.empty_like(xq), torch.empty_like(xscale), torch.empty(n, out, device="cuda")
        Q.stagq_quantize_i8(x, q, s)
        torch.cuda.synchronize()
        Q.stagq_gemm_i8(q, s, w, ws, inp, y)
        torch.cuda.synchronize()
        want.append(y)

    def chain():
        for x, y in zip(xs, got):
            Q.stagq_quantize_i8(x, xq, xscale)
            Q.stagq_gemm_i8(xq, xscale, w, ws, inp, y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(5):
        for y in got:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    Q.stagq_ops_check(0)


def test_gemv_reads_activations_of_earlier_kernels_with_plain_loads():
    # x and its inverse scale; a handle's own low values are constant and may take the read-only path
    import os
    import re
    csrc = os.path.join(os.path.dirname(Q.__file__), "csrc")
    for name in ("gemv.cu", "gemv1.cu", "kernel_common.cuh"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert "ld.global.nc" not in text, name
        assert set(re.findall(r"__ldg\((\S+)", text)) <= {"dlo", "pc.dlo"}, name


# ------------------------------------------------------------------- errors

@gpu
def test_a_call_that_cuda_refuses_leaves_no_error_behind_for_the_next():
    x, q, s = torch.ones(2, 64, dtype=F16, device="cuda"), torch.empty(2, 128, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    if torch.cuda.device_count() > 63:
        pytest.skip("device 63 exists")
    L = Q.lib()
    args = x.data_ptr(), 64, 2, 64, 0, q.data_ptr(), s.data_ptr()
    for _ in range(2):
        assert L.stagq_quantize_i8(*args, 63, None) not in (0, EINVAL)  # no such GPU
        assert L.stagq_ops_check(63) not in (0, EINVAL)
        assert float((x + 1).sum()) == 256.0  # torch looks for a pending error after its own launch
        Q.stagq_ops_check(0)
        assert L.stagq_quantize_i8(*args, 0, None) == 0
        Q.stagq_ops_check(0)
        assert (q[:, :64] == 127).all()


@gpu
def test_workspace_sizes_are_not_kept_for_every_length():
    c = Case([5], 2, 128, 64, 128, F16, width=64)
    sizes = [Q.stagq_kv_attention_workspace(c.cache, 1, n, 8, tracked=True) for n in range(1, 4097)]
    held = [v for v in vars(c.cache).values() if isinstance(v, dict)]
    assert sum(len(d) for d in held) <= 256
    assert sizes == [Q.stagq_kv_attention_workspace(c.cache, 1, n, 8, tracked=True) for n in range(1, 4097)]


# ------------------------------------------------------------------ a prompt

@gpu
def test_a_prompt_is_attended_in_steps_of_sixteen_tokens():
    n, heads, dim, page = 50, 2, 128, 16
    c = Case([n, 0], heads, dim, page, 64, F16)
    q = rnd((n, 8 * dim), 5, F16)
    out, mass = torch.empty(n, 8 * dim, dtype=F16), torch.zeros(2, heads, c.width * page, device="cuda")
    for first in range(0, n, Q.STAGQ_KV_MAX_NEW):
        m = min(Q.STAGQ_KV_MAX_NEW, n - first)
        part = torch.zeros(2 * m, 8 * dim, dtype=F16, device="cuda")
        part[:m] = q[first:first + m].cuda()
        got = torch.empty_like(part)
        lens = torch.tensor([first + m, 0], dtype=torch.int32, device="cuda")
        Q.stagq_kv_attention(c.cache, part, c.table, lens, got, n_new=m, mass=mass)
        out[first:first + m] = got[:m].cpu()
        assert not got[m:].any()
    want, p, bound, p_bound = R.attention(q.view(1, n, 8, dim), c.k[:1], c.v[:1], [n], n, dim ** -0.5)
    assert_rounded(out.view(want.shape), want, F16, bound[..., None])
    # and a rounding of the sum per call
    assert ((mass[0, :, :n].double().cpu() - p[0]).abs() <= p_bound[0] + 4 * 2.0 ** -24 * p[0]).all()
    assert not mass[1].any()
    Q.stagq_ops_check(0)


# -------------------------------------------------- shapes at the ends of the range

@gpu
@pytest.mark.parametrize("tracked", [False, True])
def test_attention_of_the_most_rows_per_kv_head(tracked):
    c = Case([300, 9], 1, 64, 16, 32, BF16)
    c.check(64, 16, tracked=tracked)  # 1024 rows


@gpu
def test_a_batch_of_thousands_of_short_sequences():
    b, heads, dim, page, budget = 3000, 2, 64, 16, 6
    lens = [i * 7 % 21 for i in range(b)]
    pool = torch.full((b * 3, Q.stagq_kv_page_bytes(heads, dim, page, 64)), 0xFF, dtype=torch.uint8, device="cuda")
    cache = Q.KVCache(pool, heads, dim, page, 64, F16)
    order = torch.randperm(b * 3, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    both = order.view(b, 3)
    table, fresh = both[:, :2], both[:, 2:]  # slices: rows 3 apart
    k, v = (rnd((b, 20, heads, dim), s, F16) for s in (1, 2))
    Q.stagq_kv_append(cache, k.view(b * 20, -1).cuda(), v.view(b * 20, -1).cuda(), table, torch.zeros(b, dtype=torch.int32, device="cuda"), 20)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = rnd((b, 2 * heads * dim), 3, F16)
    kk, vv = R.values4(k, 64), R.values4(v, 64)
    want, p, bound, p_bound = R.attention(q.view(b, 1, 2 * heads, dim), kk, vv, lens, 1, dim ** -0.5)
    mass = torch.zeros(2, b, heads, 40, device="cuda")[1, :, :, :32]  # rows further apart
    for m in (None, mass):
        out = torch.full((b, 2 * heads * dim), 3.0, dtype=F16, device="cuda")
        Q.stagq_kv_attention(cache, q.cuda(), table, n, out, mass=m)
        assert_rounded(out.view(want.shape), want, F16, bound[..., None])
    got = mass.double().cpu()
    assert ((got[..., :20] - p).abs() <= p_bound + 2.0 ** -24 * p).all() and not got[..., 20:].any()
    kept, new_lens = torch.empty(b, heads, budget, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
    new_mass = torch.full((b, heads, 12), 5.0, device="cuda")
    Q.stagq_kv_evict(cache, table, n, mass, fresh, budget, 2, kept, new_lens, new_mass[..., :8])
    assert new_lens.tolist() == [min(x, budget) for x in lens] and (new_mass[..., 8:] == 5).all()
    ko, vo = (torch.empty(b * budget, heads * dim, device="cuda") for _ in range(2))
    Q.stagq_kv_read(cache, fresh, new_lens, ko, vo, budget)
    kept, host = kept.cpu(), mass.cpu().numpy()
    for i in range(b):
        for h in range(heads):
            keep = R.keep(host[i, h], lens[i], budget, 2)
            assert kept[i, h].tolist() == keep + [-1] * (budget - len(keep)), (i, h)
    at = kept.clamp_min(0).long().permute(0, 2, 1)[..., None].expand(-1, -1, -1, dim)
    there = (kept >= 0).permute(0, 2, 1)[..., None]
    for got, values in ((ko, kk), (vo, vv)):
        assert_rounded(got.view(b, budget, heads, dim), torch.where(there, torch.gather(values, 1, at), 0.0), F32)
    Q.stagq_ops_check(0)


# ------------------------------------------------------------------- magnitudes

@gpu
@pytest.mark.parametrize("n,inp,out", [(3, 512, 200), (40, 4096, 300), (300, 512, 5000)])
def test_gemm_i8_of_activations_near_the_ends_of_bf16(n, inp, out):
    # sum * xscale alone would leave fp32 where the result does not: rows of 2^118 and of 2^-118, weights of 2^-12
    x = rnd((n, inp), n)
    x[0] *= 2.0 ** 118
    x[1] *= 2.0 ** -118
    x = x.to(BF16).cuda()
    w = (rnd((out, inp), 7) * 2.0 ** -12).to(BF16).cuda()
    row = Q.stagq_i8_row_bytes(inp)
    (xq, wq), (xs, ws) = (torch.empty(r, row, dtype=torch.int8, device="cuda") for r in (n, out)), (torch.empty(r, device="cuda") for r in (n, out))
    Q.stagq_quantize_i8(x, xq, xs)
    Q.stagq_quantize_i8(w, wq, ws)
    sums = xq[:, :inp].double() @ wq[:, :inp].double().T
    want = (sums * xs.double()[:, None] * ws.double()).cpu()
    assert want.abs().max() < 2.0 ** 127
    for dtype in (F32, BF16):
        y = torch.empty(n, out, dtype=dtype, device="cuda")
        Q.stagq_gemm_i8(xq, xs, wq, ws, inp, y)
        # the sum to fp32 and two products, the last of which is fp32's own rounding
        assert_rounded(y, want, dtype, want.abs() * (3.01 if dtype != F32 else 2.01) * 2.0 ** -24, str(dtype))
