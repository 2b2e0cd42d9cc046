"""The operators beside the GEMV at the sizes where their work is dealt out:
runs of rounds over many units, rings and accumulators used again, running
sums rescaled. Each test asserts, from the plan that the library reports, that
its sizes reach what it is there for. GPU tests need a B200."""
import pytest

torch = pytest.importorskip("torch")

import quantized_gemv_stagq_b200 as Q
from tests import operator_oracle as R
from tests.test_operators import BF16, F16, F32, Case, assert_rounded, rnd

gpu = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ plans (CPU)

def test_plan_hooks_refuse_bad_sizes():
    for args in ((0, 1, 1, 148), (1, 0, 1, 148), (1, 1, 0, 148), (1, 1, 32769, 148), (1, 1, 1, 1)):
        with pytest.raises(Q.StagqError):
            Q.stagq_debug_gemm_i8_plan(*args)
    for args in ((2, 128, 16, 128, 0, 1, 2, 1, False, 148), (2, 128, 16, 128, 1, 0, 2, 1, False, 148), (2, 96, 16, 32, 1, 1, 2, 1, False, 148),
                 (2, 128, 16, 128, 1, 1, 3, 1, False, 148), (2, 128, 16, 128, 1, 1, 2, 17, False, 148), (2, 128, 16, 128, 1, 1, 2, 1, False, 0)):
        with pytest.raises(Q.StagqError):
            Q.stagq_debug_kv_attention_plan(*args)


def test_product_plans_hold_their_invariants():
    for n in (1, 15, 16, 17, 33, 64, 65, 200, 511, 2049, 60000):
        for out in (1, 127, 129, 1285, 5003, 28672):
            for inp in (1, 128, 1285, 4096, 32768):
                width, split, pair, ctas = Q.stagq_debug_gemm_i8_plan(n, out, inp, 148)
                blocks = -(-inp // 128)
                if pair:
                    assert width in (128, 256) and split == 1 and ctas % 2 == 0 and 2 <= ctas <= 148 and n > 64
                else:
                    assert width in (16, 32, 64) and split in (1, 2, 4, 8) and split <= blocks
                    assert ctas == split * -(-out // 128) * -(-n // width)  # one tile per cluster


# ------------------------------------------------------------------- attention

class Filled(Case):
    """As Case, but written by one append: the rows past a sequence's length are NaN."""

    def __init__(self, lens, heads, dim, page, group, dtype, seed=0, k=None, v=None):
        self.lens_l, self.dtype, self.heads, self.dim, self.page, self.group = list(lens), dtype, heads, dim, page, group
        b, cap = len(lens), max(lens)
        self.width = -(-cap // page)
        n_pages = b * self.width + 3
        self.pool = torch.full((n_pages, Q.stagq_kv_page_bytes(heads, dim, page, group)), 0xFF, dtype=torch.uint8, device="cuda")
        perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.table = perm[:b * self.width].reshape(b, self.width).cuda()
        self.cache = Q.KVCache(self.pool, heads, dim, page, group, dtype)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.k_in = rnd((b, cap, heads, dim), seed + 1, dtype) if k is None else k
        self.v_in = rnd((b, cap, heads, dim), seed + 2, dtype) if v is None else v
        past = (torch.arange(cap)[None] >= torch.tensor(lens)[:, None]).cuda()
        rows = [x.cuda().masked_fill(past[:, :, None, None], float("nan")).view(b * cap, heads * dim) for x in (self.k_in, self.v_in)]
        Q.stagq_kv_append(self.cache, *rows, self.table, torch.zeros(b, dtype=torch.int32, device="cuda"), cap)
        self.k, self.v = R.values4(self.k_in, group), R.values4(self.v_in, group)

    def plan(self, q_heads, n_new, tracked):
        return Q.stagq_debug_kv_attention_plan(self.heads, self.dim, self.page, self.group, len(self.lens_l), self.width * self.page,
                                               q_heads, n_new, tracked, sms())


def dealt(lens, heads, row_blocks, ctas):
    """The even split's runs: rounds of a run (the smaller number, and whether some have one more), whether some
    unit's first part is a CTA's second or later segment, and whether some run of several units holds whole ones."""
    units, at = [], 0
    for n in lens:
        for _ in range(heads * row_blocks if n else 0):
            units.append((at, at + -(-n // 128)))
            at += -(-n // 128)
    busy = min(at, ctas)
    base, rem = divmod(at, busy)
    begins = [c * base + min(c, rem) for c in range(busy + 1)]
    later_first, whole, u = False, False, 0
    for c in range(busy):
        lo, hi = begins[c], begins[c + 1]
        while units[u][1] <= lo:
            u += 1
        i, held = u, 0
        while i < len(units) and units[i][0] < hi:
            s, e = units[i]
            if lo < s and e > hi:
                later_first = True  # begins inside the run, after other work, and goes on in the next CTA's
            held += lo <= s and e <= hi
            i += 1
        whole |= held > 0 and i - u > 1
    return base, rem, later_first, whole


RAGGED40 = [0 if i in (0, 31, 32, 39) else 1 + i * i * 97 % 2900 for i in range(40)]
RAGGED150 = [1 + i * 61 % 1000 if i % 7 else 0 for i in range(150)]
EVEN = [
    # lens, heads, query heads, new tokens, dim, page, group, type, tracked
    (RAGGED40, 3, 12, 1, 128, 64, 32, BF16, True),
    (RAGGED150, 3, 12, 1, 64, 16, 32, BF16, False),
    (RAGGED150, 3, 12, 1, 64, 16, 64, F16, True),
    ([70000], 2, 8, 1, 128, 64, 64, BF16, False),
    ([70000], 2, 8, 1, 128, 16, 128, F16, True),
    ([1, 60000], 2, 16, 1, 64, 128, 32, F16, False),          # 8 query rows per unit
    ([2500, 33, 0, 1900, 2048], 3, 48, 2, 128, 16, 64, F16, True),  # 32 rows of a KV head: 4 units
    ([3000, 7, 1900], 2, 10, 16, 64, 32, 32, BF16, True),      # 80 rows, and fewer tokens than queries
    ([4000, 129, 2999, 1], 2, 128, 1, 64, 16, 32, BF16, True),  # 64 query heads per KV head
]


@gpu
@pytest.mark.parametrize("lens,heads,q_heads,n_new,dim,page,group,dtype,tracked", EVEN)
def test_attention_dealt_out_in_runs_of_several_rounds(lens, heads, q_heads, n_new, dim, page, group, dtype, tracked):
    c = Filled(lens, heads, dim, page, group, dtype, seed=len(lens))
    rows, row_blocks, ctas, cluster = c.plan(q_heads, n_new, tracked)
    assert cluster == 0
    base, rem, later_first, whole = dealt(lens, heads, row_blocks, ctas)
    assert base > 1 and rem > 0
    assert later_first
    if len(lens) > 1 and min(-(-n // 128) for n in lens if n) < base:
        assert whole
    c.check(q_heads, n_new, tracked=tracked)


@gpu
@pytest.mark.parametrize("lens,heads,q_heads,n_new,group,dtype", [
    ([4000, 17, 2500], 2, 8, 1, 32, BF16),             # clusters of 8 with several rounds each
    (RAGGED40, 2, 8, 1, 64, F16),                      # a batch past 32
    ([3000, 5, 900], 1, 64, 1, 128, F16),              # 64 query heads of one KV head
    ([1500, 9], 2, 6, 16, 32, BF16),                   # 16 new tokens
    ([700, 130, 64, 0, 1], 33, 33, 1, 64, BF16)])      # one query row per KV head, many heads
def test_attention_by_clusters_of_several_rounds(lens, heads, q_heads, n_new, group, dtype):
    c = Filled(lens, heads, 128, 16, group, dtype, seed=3)
    rows, row_blocks, ctas, cluster = c.plan(q_heads, n_new, False)
    assert cluster >= 1 and ctas == cluster * len(lens) * heads * row_blocks
    assert max(-(-n // 128) for n in lens) > cluster  # some CTA has more than one round
    c.check(q_heads, n_new)


def _levels(tokens, seed, choices):
    """One of the choices for every 128 tokens, in random order."""
    g = torch.Generator().manual_seed(seed)
    return torch.tensor(choices)[torch.randint(len(choices), (-(-tokens // 128),), generator=g)].repeat_interleave(128)[:tokens]


@gpu
@pytest.mark.parametrize("follow", [1.0, -1.0, 3.0])
@pytest.mark.parametrize("tokens,heads,dtype", [(4000, 2, BF16), (72000, 4, BF16), (72000, 4, F16)])
def test_running_sums_are_rescaled_as_scores_and_scales_rise(tokens, heads, dtype, follow):
    """V's scale and the scores change by up to 2^12 and 2^(12 follow) from one
    of a warp's tiles to the next, in either order, so that its sums are
    rescaled with something in them. follow = 1: large V has small weights.

    Bound: twice the scores' error on sum p |V|; and what rounding p s to fp16
    parts cuts, below 2^-24 of the parts' unit, which is at least 2^-6 of the
    largest scale s that the warp has met: 2^-30 s per token and unit of the
    code's distance from 8, for the tokens of a warp, whose weights sum to 1 at
    least."""
    dim, group = 64, 32
    a = _levels(tokens, tokens, [-6.0, -3.0, 0.0, 3.0, 6.0])
    k = rnd((1, tokens, heads, dim), 1) * 0.5
    v = (1 + 0.3 * rnd((1, tokens, heads, dim), 2)) * torch.exp2(a)[None, :, None, None]
    k[..., 0] = -a[None, :, None] * follow * 0.6931 * dim ** 0.5 / 16
    q = rnd((1, heads * 4 * dim), 3).view(1, 1, heads * 4, dim)
    q[..., 0] = 16.0
    q = q.to(dtype)
    c = Filled([tokens], heads, dim, 16, group, dtype, k=k.to(dtype), v=v.to(dtype))
    rows, row_blocks, ctas, cluster = c.plan(heads * 4, 1, False)
    per_cta = -(-tokens // 128) / cluster if cluster else dealt([tokens], heads, row_blocks, ctas)[0]
    assert per_cta >= 3.9  # tiles of a warp
    got = c.attend(q.view(1, -1).cuda(), 1)
    want, _, bound, _ = R.attention(q, c.k, c.v, [tokens], 1, dim ** -0.5)
    weighted, _, _, _ = R.attention(q, c.k, c.v.abs(), [tokens], 1, dim ** -0.5)
    err = bound / (2 * c.v.abs().max())
    scale_max = R.rounded4(c.v_in, group)[1].max()
    extra = 2 * err[..., None] * weighted + 32 * (per_cta + 2) * 2.0 ** -27 * scale_max
    assert_rounded(got.view(want.shape), want, dtype, extra, "out")
    Q.stagq_ops_check(0)


@gpu
@pytest.mark.parametrize("first,last", [(-80.0, 50.0), (50.0, -80.0), (-120.0, 100.0)])
def test_scales_of_v_more_than_2_to_the_126_apart(first, last):
    tokens, heads = 4000, 2
    a = torch.where(torch.arange(tokens) < 2000, first, last)
    a[::256] = last  # and in the middle of the first half
    v = (rnd((1, tokens, heads, 128), 2).double() * torch.exp2(a.double())[None, :, None, None]).to(BF16)
    Filled([tokens], heads, 128, 16, 64, BF16, v=v).check(8, 1)
    Filled([tokens], heads, 128, 16, 64, BF16, v=v).check(8, 2, tracked=True)


@gpu
@pytest.mark.parametrize("group,dtype", [(128, F16), (32, BF16)])
@pytest.mark.parametrize("k", [6, 10, 13])
def test_attention_of_queries_with_one_large_channel(k, group, dtype):
    # one channel 2^k times the others: what the codes' products drop is relative to the row's largest
    c = Filled([700, 500], 2, 128, 16, group, dtype, seed=3)
    q = rnd((2, 128 * 8), 3) * 2.0 ** -6
    q.view(2, 8, 128)[:, :, 5] = 2.0 ** (k - 5)
    q.view(2, 8, 128)[:, 1::2, 5] *= -1
    scale = 64 * 128 ** -0.5 * 2.0 ** -max(0, k - 5)
    c.check(8, 1, q=q.to(dtype), scale=scale)
    c.check(8, 1, q=q.to(dtype), scale=scale, tracked=True)


@gpu
def test_repeated_calls_give_the_same_bits():
    # of long sequences shared by all CTAs, into outputs, masses and workspaces of their own, on two streams
    c = Filled([30000, 0, 11111], 3, 128, 64, 64, BF16)
    q = rnd((3, 12 * 128), 5, BF16).cuda()
    outs = []
    for s in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        out, mass = torch.full_like(q, 3.0), torch.zeros(3, 3, c.width * 64, device="cuda")
        plain = torch.full_like(q, 5.0)
        torch.cuda.synchronize()
        Q.stagq_kv_attention(c.cache, q, c.table, c.lens, out, mass=mass, stream=s)
        Q.stagq_kv_attention(c.cache, q, c.table, c.lens, plain, stream=s)
        outs.append((out, mass, plain))
    torch.cuda.synchronize()
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)
    Q.stagq_ops_check(0)


# --------------------------------------------------------------------- product

PAIRS = [
    # n, in, out, channels of a tile, tiles per pair at least
    (60001, 2100, 100, 128, 4), (45000, 1285, 77, 128, 3), (1500, 5003, 1285, 128, 1), (1001, 17920, 2000, 128, 1),
    (2049, 5003, 4101, 256, 3), (3001, 2100, 5001, 256, 4), (4100, 1285, 6000, 256, 6), (520, 5003, 4000, 256, 1)]


@gpu
@pytest.mark.parametrize("n,inp,out,width,tiles", PAIRS)
def test_gemm_i8_pairs_use_their_rings_and_accumulators_again(n, inp, out, width, tiles):
    plan = Q.stagq_debug_gemm_i8_plan(n, out, inp, sms())
    per_pair = -(-(-(-n // 256) * -(-out // width)) // (plan[3] // 2))
    assert plan[0] == width and plan[2] == 1 and per_pair >= tiles
    assert per_pair * -(-inp // 128) > 2 * 8  # K blocks of a CTA, against at most 8 stages
    g = torch.Generator(device="cuda").manual_seed(n)
    row = Q.stagq_i8_row_bytes(inp)
    a, b = (torch.zeros(r, row, dtype=torch.int8, device="cuda") for r in (n, out))
    a[:, :inp] = torch.randint(-128, 128, (n, inp), generator=g, device="cuda", dtype=torch.int8)
    b[:, :inp] = torch.randint(-128, 128, (out, inp), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.exp2(torch.randint(-9, -5, (n,), generator=g, device="cuda").float())  # powers of two: one rounding, of the sum
    ws = torch.exp2(torch.randint(-9, -5, (out,), generator=g, device="cuda").float())
    want = (a.double() @ b.double().T).float() * xs[:, None] * ws
    for dtype in (F32, F16, BF16):
        for first in (0, 1):  # rows of y on 16 bytes where `out` allows it, and not
            whole = torch.full((n, out + 8), 7.0, dtype=dtype, device="cuda")
            Q.stagq_gemm_i8(a, xs, b, ws, inp, whole[:, first:first + out])
            assert torch.equal(whole[:, first:first + out], want.to(dtype)), (dtype, first)
            assert (whole[:, :first] == 7).all() and (whole[:, first + out:] == 7).all()
    Q.stagq_ops_check(0)


# -------------------------------------------------------------------- launches

@gpu
@pytest.mark.parametrize("lens,tracked", [([777], False), ([4000, 9], False), ([70000], False), ([777], True)])
def test_launches_that_the_benchmark_counts(lens, tracked):
    runtime = pytest.importorskip("cuda.bindings.runtime")
    import bench
    c = Filled(lens, 2, 128, 64, 128, F16)
    q = rnd((len(lens), 8 * 128), 5, F16).cuda()
    need = Q.stagq_kv_attention_workspace(c.cache, len(lens), c.width * 64, 8, 1, tracked)
    ws, out = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    mass = torch.zeros(len(lens), 2, c.width * 64, device="cuda") if tracked else None
    k = torch.zeros(len(lens), 2 * 128, dtype=F16, device="cuda")
    x, xq, xs = torch.zeros(5, 256, dtype=F16, device="cuda"), torch.empty(5, 256, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    y = torch.empty(5, 5, device="cuda")

    def attention():
        Q.stagq_kv_attention(c.cache, q, c.table, c.lens, out, mass=mass, workspace=ws)

    def linear():
        Q.stagq_quantize_i8(x, xq, xs)
        Q.stagq_gemm_i8(xq, xs, xq, xs, 256, y)

    starts = c.lens - 1
    for body, kernels in ((attention, bench._attention_launches(need)), (linear, 2),
                          (lambda: Q.stagq_kv_append(c.cache, k, k, c.table, starts, 1), 1)):
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(graph):
            body()
        status, _, nodes = runtime.cudaGraphGetNodes(graph.raw_cuda_graph(), 0)
        assert status == runtime.cudaError_t.cudaSuccess
        assert nodes == kernels


# --------------------------------------------- scales that a row does not see, or hardly

@gpu
@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("q_heads,tokens", [(4, 40), (4, 333), (16, 333)])
@pytest.mark.parametrize("dim,group,dtype", [(128, 128, F16), (128, 32, BF16), (64, 64, BF16)])
def test_an_extreme_v_that_a_row_does_not_see_costs_it_nothing(dim, group, dtype, q_heads, tokens, tracked):
    # the newest of three tokens holds the type's largest values: the two before it do not see them
    v = rnd((1, tokens, 2, dim), 4, dtype)
    v[0, -1, :, ::2], v[0, -1, :, 1::2] = torch.finfo(dtype).max / 4, torch.finfo(dtype).min / 4
    c = Filled([tokens], 2, dim, 16, group, dtype, v=v)
    q = rnd((3, q_heads * dim), 5, dtype)
    got = c.attend(q.cuda(), 3, torch.zeros(1, 2, c.width * 16, device="cuda") if tracked else None)
    want, _, bound, _ = R.attention(q.view(1, 3, q_heads, dim), c.k, c.v, [tokens], 3, dim ** -0.5)
    assert_rounded(got.view(want.shape), want, dtype, bound[..., None], "out")
    Q.stagq_ops_check(0)


@gpu
@pytest.mark.parametrize("at", [0, 700, 1499])
@pytest.mark.parametrize("n_new,tracked", [(1, False), (2, True)])
@pytest.mark.parametrize("dtype,large", [(F16, 13.0), (BF16, 13.0), (BF16, 34.0)])
def test_a_large_v_of_small_weight_leaves_the_others_their_bits(dtype, large, n_new, tracked, at):
    """One token's V is 2^13 or 2^34 times the others', and its weight 2^-40 for every second query row while the others attend
    to it alone. Bound: twice the scores' error on sum p |V|, and what the parts of p s cut: 2^-30, per token and unit of
    the code's distance from 8, of a scale that follows max p s within 2^8."""
    tokens, heads, dim, group = 1500, 2, 128, 64
    k, v = rnd((1, tokens, heads, dim), 1) * 0.3, 1 + 0.3 * rnd((1, tokens, heads, dim), 2)
    k[..., 0], k[0, at, :, 0] = 0.0, 20.0
    v[0, at] *= 2.0 ** large
    q = rnd((n_new, heads * 4, dim), 3)
    q[:, 0::2, 0], q[:, 1::2, 0] = 16.0, -16.0  # scores of the large token: +28 and -28 nats
    q = q.to(dtype)
    c = Filled([tokens + 2], heads, dim, 16, group, dtype, k=torch.cat([k, rnd((1, 2, heads, dim), 8) * 0.3], 1).to(dtype),
               v=torch.cat([v, 1 + 0.3 * rnd((1, 2, heads, dim), 9)], 1).to(dtype))
    n = tokens + 2
    got = c.attend(q.view(n_new, -1).cuda(), n_new, torch.zeros(1, heads, c.width * 16, device="cuda") if tracked else None)
    scale = dim ** -0.5
    want, _, bound, _ = R.attention(q[None], c.k, c.v, [n], n_new, scale)
    weighted, _, _, _ = R.attention(q[None], c.k, c.v.abs(), [n], n_new, scale)
    err = bound / (2 * c.v.abs().max())
    s = R.rounded4(c.v_in, group)[1].amax(-1)[0].cpu()  # [tokens, heads]
    scores = torch.einsum("jhpd,thd->jhpt", q.double().view(n_new, heads, 4, dim), c.k[0]) * scale
    ps = (torch.softmax(scores, -1) * s.T[None, :, None]).amax(-1).view(1, n_new, heads * 4, 1)
    extra = 2 * err[..., None] * weighted + n * 2.0 ** -19 * ps
    assert_rounded(got.view(want.shape), want, dtype, extra, "out")
    Q.stagq_ops_check(0)
