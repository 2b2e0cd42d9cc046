"""The operators beside the GEMV (8-bit linear, 4-bit cache) against plain
forms in 64 bits, and their refusals. GPU tests need a B200."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_gemv_stagq_b200 as Q
from quantized_gemv_stagq_b200 import synth
from tests import operator_oracle as R

gpu = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
EINVAL, EFORMAT = 1, 2


def rnd(shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_rounded(got, want, dtype, extra=0.0, what=""):
    """got (of dtype) is `want` (float64) rounded once, after an error of at most `extra`."""
    got = got.to(torch.float64).cpu()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # a subnormal's step
    limit = want.abs() * half_step(dtype) * (1 + 2 ** -8) + extra * (1 + half_step(dtype)) + tiny
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaNs elsewhere"
    off = ((got - want).abs() - limit).nan_to_num(0.0)
    assert float(off.max() if off.numel() else 0.0) <= 0, f"{what}: off by {float(off.max()):.3e} more than allowed"


# ------------------------------------------------------------------ refusals (CPU)

def _fake(n=1):
    return ctypes.c_void_p(4096 * n)  # never dereferenced: every call below is refused


def test_i8_refuses_bad_arguments_before_any_device_work():
    L = Q.lib()
    assert Q.stagq_i8_row_bytes(1) == 128 and Q.stagq_i8_row_bytes(128) == 128 and Q.stagq_i8_row_bytes(129) == 256
    for inp in (0, -1, 32769):
        assert L.stagq_i8_row_bytes(inp) == -1
        with pytest.raises(ValueError):
            Q.stagq_i8_row_bytes(inp)
    ok = dict(x=_fake(), xs=64, n=2, inp=64, flags=0, q=_fake(2), s=_fake(3), dev=0)
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(n=0), dict(n=-1), dict(inp=0), dict(inp=40000), dict(xs=63),
                dict(flags=1), dict(flags=32), dict(q=ctypes.c_void_p(4097)), dict(dev=-1), dict(dev=64)):
        a = {**ok, **bad}
        assert L.stagq_quantize_i8(a["x"], a["xs"], a["n"], a["inp"], a["flags"], a["q"], a["s"], a["dev"], None) == EINVAL, bad
    ok = dict(xq=_fake(), xs=_fake(2), n=2, wq=_fake(3), ws=_fake(4), out=8, inp=64, y=_fake(5), ys=8, flags=0, dev=0)
    for bad in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y=None), dict(n=0), dict(out=0), dict(inp=0),
                dict(inp=32769), dict(ys=7), dict(flags=2), dict(flags=1 | 16), dict(xq=ctypes.c_void_p(4104)),
                dict(wq=ctypes.c_void_p(4104)), dict(dev=-1), dict(n=2 ** 31 - 1, out=2 ** 31 - 1, ys=2 ** 31)):
        a = {**ok, **bad}
        assert L.stagq_gemm_i8(a["xq"], a["xs"], a["n"], a["wq"], a["ws"], a["out"], a["inp"], a["y"], a["ys"], a["flags"],
                               a["dev"], None) == EINVAL, bad


def _cache_c(**kw):
    f = dict(pages=4096, n_pages=4, heads=2, dim=128, page=16, group=128, flags=0, device=0)
    f.update(kw)
    return Q._KvCache(*f.values())


BAD_CACHES = [dict(dim=96), dict(dim=256), dict(group=16), dict(group=256), dict(dim=64, group=128), dict(page=8), dict(page=48),
              dict(page=2048), dict(heads=0), dict(heads=5000), dict(flags=1), dict(device=-1), dict(device=64)]
BAD_TABLES = [dict(pages=None), dict(batch=0), dict(width=0), dict(row_stride=3), dict(width=2 ** 27, row_stride=2 ** 27)]


def test_kv_refuses_bad_arguments_before_any_device_work():
    L = Q.lib()
    r = ctypes.byref
    good, tab = _cache_c(), dict(pages=8192, row_stride=4, batch=2, width=4)
    table = Q._KvTable(*tab.values())
    assert L.stagq_kv_page_bytes(r(good)) == 2 * 2 * 16 * (64 + 4)
    p, row = _fake(), 256

    def rows(c=good, t=table, starts=p, k=p, ks=row, v=p, vs=row, n=1):
        return L.stagq_kv_append(r(c), r(t), starts, k, ks, v, vs, n, None), L.stagq_kv_read(r(c), r(t), starts, starts, k, ks, v, vs, n, 0, None)

    def attend(c=good, t=table, lens=p, max_len=64, q=p, qs=1024, q_heads=8, n_new=1, scale=0.1, out=p, outs=1024, mass=None,
               mb=128, mh=64, ws=p, wb=1 << 40):
        return L.stagq_kv_attention(r(c), r(t), lens, max_len, q, qs, q_heads, n_new, scale, out, outs, mass, mb, mh, ws, wb, None)

    def evict(c=good, t=table, lens=p, max_len=64, mass=p, mb=128, mh=64, budget=8, recent=2, f=table, kept=p, nl=p, nm=p, nb=128,
              nh=64, cap=64):
        return L.stagq_kv_evict(r(c), r(t), lens, max_len, mass, mb, mh, budget, recent, r(f), kept, nl, nm, nb, nh, cap, None)

    for kw in BAD_CACHES:
        c = _cache_c(**kw)
        assert L.stagq_kv_page_bytes(r(c)) == -1, kw
        assert rows(c=c) == (EINVAL, EINVAL) and attend(c=c) == EINVAL and evict(c=c) == EINVAL, kw
        assert L.stagq_kv_attention_workspace(r(c), 1, 64, 8, 1, 0) == -1
    for kw in (dict(pages=None), dict(pages=4100), dict(n_pages=0)):
        c = _cache_c(**kw)
        assert rows(c=c) == (EINVAL, EINVAL) and attend(c=c) == EINVAL and evict(c=c) == EINVAL, kw
    for kw in BAD_TABLES:
        t = Q._KvTable(*{**tab, **kw}.values())
        assert rows(t=t) == (EINVAL, EINVAL) and attend(t=t) == EINVAL and evict(t=t) == EINVAL and evict(f=t) == EINVAL, kw
    for kw in (dict(k=None), dict(v=None), dict(ks=255), dict(vs=255), dict(ks=2 ** 31), dict(vs=2 ** 31), dict(n=0), dict(n=2 ** 30 + 1)):
        assert rows(**kw) == (EINVAL, EINVAL), kw
    assert rows(starts=None)[0] == EINVAL
    assert L.stagq_kv_read(r(good), r(table), None, None, p, row, p, row, 1, 2, None) == EINVAL
    for kw in (dict(lens=None), dict(q=None), dict(out=None), dict(max_len=0), dict(max_len=65), dict(q_heads=0), dict(q_heads=7),
               dict(q_heads=130), dict(n_new=0), dict(n_new=17), dict(qs=1023), dict(outs=1023), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(mass=p, mh=63), dict(mass=p, mb=127)):
        assert attend(**kw) == EINVAL, kw
    small = Q._KvTable(8192, 4, 3, 4)
    for kw in (dict(lens=None), dict(mass=None), dict(kept=None), dict(nl=None), dict(nm=None), dict(max_len=0), dict(max_len=65),
               dict(budget=0), dict(budget=65), dict(recent=-1), dict(recent=9), dict(cap=7), dict(mh=63), dict(nh=63), dict(mb=127),
               dict(nb=127), dict(f=small)):
        assert evict(**kw) == EINVAL, kw
    assert L.stagq_ops_check(-1) == EINVAL and L.stagq_ops_check(64) == EINVAL
    with pytest.raises(ValueError):
        Q.stagq_kv_page_bytes(2, 96, 16, 32)


def test_binding_refuses_tensors_off_the_gpu():
    x, q = torch.zeros(2, 64, dtype=F16), torch.zeros(2, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        Q.stagq_quantize_i8(x, q, torch.zeros(2))
    with pytest.raises(TypeError):
        Q.stagq_quantize_i8(x.numpy(), q, torch.zeros(2))
    with pytest.raises(ValueError):
        Q.stagq_gemm_i8(q, torch.zeros(2), q, torch.zeros(2), 64, torch.zeros(2, 2, dtype=F16))
    with pytest.raises(ValueError):
        Q.KVCache(torch.zeros(Q.stagq_kv_page_bytes(2, 64, 16, 32), dtype=torch.uint8), 2, 64, 16, 32, F16)


# --------------------------------------------------------------- 8-bit linear (GPU)

@gpu
@pytest.mark.parametrize("n,inp,dtype", [(1, 1, F16), (1, 4096, F16), (3, 127, F16), (5, 129, BF16), (7, 5003, BF16), (2, 17920, F16),
                                         (1, 32768, BF16), (300, 640, F16)])
def test_quantize_i8_equals_the_formula(n, inp, dtype):
    x = rnd((n, inp), inp, dtype)
    x[0, 0] = 3.5
    if n > 2:
        x[1] = 0.0                                             # a row of zeros
        x[2] = x[2] * (2.0 ** -20 if dtype == F16 else 1e-30)  # a tiny one
    if n > 4:  # every quotient a tie: 127 x / a = k + 1/2 for x = (2 k + 1) a / 254
        k = torch.arange(inp) % 126
        x[3] = (2 * k + 1).to(dtype) / 2
        x[3, 0] = 127.0 if inp < 5000 else 63.5
        x[4] = 0.0
        x[4, inp - 1] = torch.finfo(dtype).max
        x[4, 0] = -torch.finfo(dtype).max / 2
    row = Q.stagq_i8_row_bytes(inp)
    q = torch.full((n, row), 99, dtype=torch.int8, device="cuda")
    scale = torch.empty(n, device="cuda")
    Q.stagq_quantize_i8(x.cuda(), q, scale)
    want, ws = R.quantize_i8(x)
    assert torch.equal(q[:, :inp].cpu().double(), want)
    assert not q[:, inp:].any()
    assert torch.equal(scale.cpu(), x.abs().amax(1).float() / 127)
    assert_rounded(scale, ws, F32)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_quantize_i8_rows_apart_unaligned_and_not_finite(dtype):
    base = rnd((6, 700), 3, dtype).cuda()
    q, scale = torch.empty(6, 256, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    for first in (0, 1, 8):  # slices whose rows do and do not start on 16 bytes
        x = base[:, first:first + 200]
        Q.stagq_quantize_i8(x, q, scale)
        assert torch.equal(q[:, :200].cpu().double(), R.quantize_i8(x.cpu())[0])
    x = base[:, :200].contiguous()
    x[1, 5], x[2, 199], x[3, 0] = float("nan"), float("inf"), float("-inf")
    Q.stagq_quantize_i8(x, q, scale)
    want, ws = R.quantize_i8(x.cpu())
    assert torch.equal(q[:, :200].cpu().double(), want)
    assert torch.isnan(scale).cpu().tolist() == [False, True, True, True, False, False]
    w = torch.randint(-127, 128, (64, 256), dtype=torch.int8, device="cuda")
    w[:, 200:] = 0
    y = torch.empty(6, 64, dtype=dtype, device="cuda")
    Q.stagq_gemm_i8(q, scale, w, torch.ones(64, device="cuda"), 200, y)
    assert torch.isnan(y).all(1).cpu().tolist() == [False, True, True, True, False, False]
    assert torch.isfinite(y[[0, 4, 5]].float()).all()


def _i8(n, inp, out, seed, extreme=False):
    g = torch.Generator().manual_seed(seed)
    row = Q.stagq_i8_row_bytes(inp)
    a, b = torch.zeros(n, row, dtype=torch.int8), torch.zeros(out, row, dtype=torch.int8)
    if extreme:
        a[:, :inp], b[:, :inp] = -128, -128
    else:
        a[:, :inp] = torch.randint(-128, 128, (n, inp), generator=g, dtype=torch.int8)
        b[:, :inp] = torch.randint(-128, 128, (out, inp), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(n, generator=g) + 0.01, torch.rand(out, generator=g) * 0.01
    want = (a[:, :inp].double() @ b[:, :inp].double().T) * xs.double()[:, None] * ws.double()
    return a.cuda(), xs.cuda(), b.cuda(), ws.cuda(), want


GEMM = [(1, 1, 1), (1, 128, 128), (2, 4096, 300), (16, 1024, 129), (17, 2048, 1000), (31, 130, 77), (33, 8192, 257), (64, 5003, 640),
        (65, 257, 4096), (100, 1536, 200), (128, 128, 128), (129, 640, 384), (255, 1000, 513), (300, 512, 5000), (700, 384, 2600),
        (1, 32768, 256), (40, 32768, 64), (2049, 256, 2500)]


@gpu
@pytest.mark.parametrize("n,inp,out", GEMM)
def test_gemm_i8_against_64_bits(n, inp, out):
    a, xs, b, ws, want = _i8(n, inp, out, n + inp)
    for dtype in (F32, F16, BF16):
        y = torch.full((n, out), 7.0, dtype=dtype, device="cuda")
        Q.stagq_gemm_i8(a, xs, b, ws, inp, y)
        # fp32: the sum to fp32 and two products, a rounding each; then the output's
        extra = want.abs() * (3.01 * 2.0 ** -24 if dtype != F32 else 2.01 * 2.0 ** -24)
        assert_rounded(y, want, dtype, extra, f"{n}x{inp}x{out} {dtype}")
    Q.stagq_ops_check(0)


@gpu
def test_gemm_i8_sums_are_exact_at_their_largest():
    a, xs, b, ws, want = _i8(20, 32768, 130, 1, extreme=True)
    y = torch.empty(20, 130, device="cuda")
    Q.stagq_gemm_i8(a, xs, b, ws, 32768, y)
    assert_rounded(y, want, F32, want.abs() * 2.01 * 2.0 ** -24)


@gpu
def test_gemm_i8_rows_apart_and_neighbours_untouched():
    a, xs, b, ws, want = _i8(70, 300, 140, 5)
    whole = torch.full((72, 200), 5.0, dtype=F16, device="cuda")
    Q.stagq_gemm_i8(a, xs, b, ws, 300, whole[1:71, 33:173])
    assert_rounded(whole[1:71, 33:173], want, F16, want.abs() * 3.01 * 2.0 ** -24)
    whole[1:71, 33:173] = 5.0
    assert (whole == 5.0).all()


@gpu
def test_gemm_i8_a_row_does_not_depend_on_the_batch():
    a, xs, b, ws, _ = _i8(600, 4096, 520, 9)
    y = torch.empty(600, 520, device="cuda")
    Q.stagq_gemm_i8(a, xs, b, ws, 4096, y)
    for n in (1, 16, 20, 64, 80, 200):
        z = torch.empty(n, 520, device="cuda")
        Q.stagq_gemm_i8(a[:n], xs[:n], b, ws, 4096, z)
        assert torch.equal(z, y[:n]), n


@gpu
def test_gemm_i8_binding_refuses_what_does_not_fit():
    a, xs, b, ws, _ = _i8(4, 300, 140, 5)
    y = torch.empty(4, 140, device="cuda", dtype=F16)
    for args in ((a[:, :256], xs, b, ws, 300, y), (a, xs[:3], b, ws, 300, y), (a, xs, b[:, :256], ws, 300, y), (a, xs, b, ws[:1], 300, y),
                 (a, xs, b, ws, 500, y), (a, xs, b, ws, 300, y[:3]), (a, xs, b, ws, 300, y.t().contiguous().t()),
                 (a, xs.cpu(), b, ws, 300, y)):
        with pytest.raises(ValueError):
            Q.stagq_gemm_i8(*args)
    for args in ((a.float(), xs, b, ws, 300, y), (a, xs.half(), b, ws, 300, y), (a, xs, b, ws, 300, y.double())):
        with pytest.raises(TypeError):
            Q.stagq_gemm_i8(*args)
    with pytest.raises(ValueError):
        Q.stagq_quantize_i8(torch.zeros(4, 300, dtype=F16, device="cuda").t(), a, xs)


# ----------------------------------------------------------------- 4-bit cache (GPU)

class Case:
    """A pool with shuffled pages, filled by stagq_kv_append; k, v: the values
    that the cache stands for (float64, CPU)."""

    def __init__(self, lens, heads=2, dim=128, page=16, group=128, dtype=F16, seed=0, width=None, junk=0xFF, k=None, v=None, spare=3):
        self.lens_l, self.dtype, self.heads, self.dim, self.page, self.group = list(lens), dtype, heads, dim, page, group
        b, cap = len(lens), max(1, max(lens))
        self.width = width or -(-cap // page)
        n_pages = b * self.width + spare
        # what no call wrote is 0xFF bytes: NaN scales and lowest values
        self.pool = torch.full((n_pages, Q.stagq_kv_page_bytes(heads, dim, page, group)), junk, dtype=torch.uint8, device="cuda")
        perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.table = perm[:b * self.width].reshape(b, self.width).cuda()
        self.unused = perm[b * self.width:]
        self.cache = Q.KVCache(self.pool, heads, dim, page, group, dtype)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.k_in = rnd((b, cap, heads, dim), seed + 1, dtype) if k is None else k
        self.v_in = rnd((b, cap, heads, dim), seed + 2, dtype) if v is None else v
        for i, n in enumerate(lens):  # each sequence by itself: only its own tokens are written
            if n:
                starts = torch.full((b,), -1, dtype=torch.int32, device="cuda")
                starts[i] = 0
                rows = [torch.zeros(b * n, heads * dim, dtype=dtype) for _ in range(2)]
                rows[0].view(b, n, heads, dim)[i], rows[1].view(b, n, heads, dim)[i] = self.k_in[i, :n], self.v_in[i, :n]
                Q.stagq_kv_append(self.cache, rows[0].cuda(), rows[1].cuda(), self.table, starts, n)
        self.k, self.v = R.values4(self.k_in, group), R.values4(self.v_in, group)

    def attend(self, q, n_new, mass=None, scale=None, **kw):
        out = torch.full_like(q, 3.0)
        Q.stagq_kv_attention(self.cache, q, self.table, self.lens, out, n_new=n_new, mass=mass, scale=scale, **kw)
        return out

    def check(self, q_heads, n_new, seed=7, q=None, scale=None, tracked=False, **kw):
        b = len(self.lens_l)
        q = rnd((b * n_new, q_heads * self.dim), seed, self.dtype) if q is None else q
        mass0 = torch.rand(b, self.heads, self.width * self.page).cuda() if tracked else None
        mass = mass0.clone() if tracked else None
        got = self.attend(q.cuda(), n_new, mass, scale, **kw)
        sc = self.dim ** -0.5 if scale is None else scale
        out, p, bound, p_bound = R.attention(q.view(b, n_new, q_heads, self.dim), self.k, self.v, self.lens_l, n_new, sc)
        assert_rounded(got.view(out.shape), out, self.dtype, bound[..., None], "out")
        if tracked:
            for i, n in enumerate(self.lens_l):
                want = mass0[i, :, :n].double().cpu() + p[i, :, :n]
                d = (mass[i, :, :n].double().cpu() - want).abs()
                assert (d <= p_bound[i, :, :n] + 2.0 ** -24 * want).all()  # and the rounding of the last sum
                assert torch.equal(mass[i, :, n:], mass0[i, :, n:])
        Q.stagq_ops_check(0)
        return got


FORMATS = [(128, 128, 16, F16), (128, 64, 32, BF16), (128, 32, 64, F16), (64, 64, 16, BF16), (64, 32, 128, F16)]


@gpu
@pytest.mark.parametrize("dim,group,page,dtype", FORMATS)
def test_append_writes_the_documented_bytes(dim, group, page, dtype):
    heads, lens = 3, [37, 1]
    k, v = rnd((2, 37, heads, dim), 1, dtype), rnd((2, 37, heads, dim), 2, dtype, 0.1)
    k[0, 0] = 1.25                                     # constant groups
    k[0, 1, 0, 5], v[0, 2, 1, 0], v[0, 3, 2, dim - 1] = float("nan"), float("inf"), float("-inf")
    k[0, 4] *= 2.0 ** -18 if dtype == F16 else 1e-36   # subnormal scales
    k[0, 5, :, ::2], k[0, 5, :, 1::2] = torch.finfo(dtype).max, torch.finfo(dtype).min
    k[0, 6] = (torch.arange(dim) % 31).to(dtype) / 2   # quotients (x - lo) / s that are ties: s = 1, x = n / 2
    c = Case(lens, heads, dim, page, group, dtype, k=k, v=v)
    raw = c.pool.cpu().numpy().reshape(-1, heads, 2, page * (dim // 2 + 4 * dim // group))
    untouched = np.ones(raw.shape, bool)
    ng, bits = dim // group, torch.int16
    for b, n in enumerate(lens):
        for t in range(n):
            pid, slot = int(c.table[b, t // page]), t % page
            for which, x in enumerate((k, v)):
                u, s, lo = R.rounded4(x[b, t], group)
                codes = R.code_bytes(u.flatten(-2), which)
                meta = torch.stack([s, lo], -1).to(dtype)
                at = slot * dim // 2
                assert np.array_equal(raw[pid, :, which, at:at + dim // 2], codes), (b, t, which)
                m0 = page * dim // 2 + slot * 4 * ng
                got = torch.from_numpy(raw[pid, :, which, m0:m0 + 4 * ng].copy()).view(dtype).view(heads, ng, 2)
                assert torch.equal(torch.isnan(got), torch.isnan(meta)) and torch.equal(got.nan_to_num(0), meta.nan_to_num(0)), (b, t, which)
                untouched[pid, :, which, at:at + dim // 2] = untouched[pid, :, which, m0:m0 + 4 * ng] = False
    assert (raw[untouched] == 0xFF).all()


@gpu
@pytest.mark.parametrize("dim,group,page,dtype", FORMATS)
def test_read_gives_the_values_back(dim, group, page, dtype):
    heads, lens, n = 2, [50, 0, 17], 20
    c = Case(lens, heads, dim, page, group, dtype)
    for starts in (None, [40, 3, -2]):
        st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
        for out in (dtype, F32):
            k, v = (torch.full((3 * n, heads * dim), 9.0, dtype=out, device="cuda") for _ in range(2))
            Q.stagq_kv_read(c.cache, c.table, c.lens, k, v, n, starts=st)
            for got, x in ((k, c.k), (v, c.v)):
                want = torch.zeros(3, n, heads, dim, dtype=torch.float64)
                for b in range(3):
                    for i in range(n):
                        p = (starts[b] if starts else 0) + i
                        if 0 <= p < lens[b]:
                            want[b, i] = x[b, p]
                assert_rounded(got.view(want.shape), want, out)
    Q.stagq_ops_check(0)


@gpu
def test_append_takes_slices_of_a_stacked_result_and_unaligned_rows():
    heads, dim, lens = 2, 64, [5, 9]
    for first in (0, 8, 1):  # rows on 16 bytes, and not
        qkv = rnd((2 * 9, first + 3 * heads * dim + 7), first, F16).cuda()
        c = Case(lens, heads, dim, 16, 32, F16)
        k, v = (qkv[:, first + i * heads * dim:first + (i + 1) * heads * dim] for i in (1, 2))
        Q.stagq_kv_append(c.cache, k, v, c.table, torch.zeros(2, dtype=torch.int32, device="cuda"), 9)
        ko, vo = (torch.empty(18, heads * dim, device="cuda") for _ in range(2))
        Q.stagq_kv_read(c.cache, c.table, None, ko, vo, 9)
        assert_rounded(ko, R.values4(k.cpu().view(18, heads, dim), 32).flatten(1), F32)
        assert_rounded(vo, R.values4(v.cpu().view(18, heads, dim), 32).flatten(1), F32)


@gpu
def test_bad_pages_and_positions_are_reported_and_written_nowhere():
    c = Case([20, 20], 2, 64, 16, 64, F16)
    before = c.pool.clone()
    k = torch.ones(2 * 20, 2 * 64, dtype=F16, device="cuda")
    bad = c.table.clone()
    bad[0] = torch.tensor([-1, c.pool.shape[0]], dtype=torch.int32)
    starts = torch.tensor([0, -1], dtype=torch.int32, device="cuda")
    for table, s in ((bad, starts), (c.table, starts + 32)):  # bad numbers; positions past the table (and 31: the last one inside)
        s = s.clone()
        s[1] = -1
        Q.stagq_kv_append(c.cache, k, k, table, s, 20)
        with pytest.raises(Q.StagqError) as e:
            Q.stagq_ops_check(0)
        assert e.value.status == EFORMAT
        assert torch.equal(c.pool, before)
        Q.stagq_ops_check(0)  # reported once
    ko, vo = (torch.full((40, 128), 9.0, dtype=F16, device="cuda") for _ in range(2))
    Q.stagq_kv_read(c.cache, bad, c.lens, ko, vo, 20)
    with pytest.raises(Q.StagqError):
        Q.stagq_ops_check(0)
    assert not ko[:20].any() and ko[20:].any()
    # attention: the tokens of a bad page count as unseen, the other sequence is right
    q = rnd((2, 4 * 64), 3, F16).cuda()
    good = c.attend(q, 1)
    bad[0, 0] = c.table[0, 0]
    out = torch.empty_like(q)
    Q.stagq_kv_attention(c.cache, q, bad, c.lens, out)
    with pytest.raises(Q.StagqError):
        Q.stagq_ops_check(0)
    assert torch.equal(out[1], good[1])
    want, _, bound, _ = R.attention(q.cpu().view(2, 1, 4, 64), c.k, c.v, [16, 20], 1, 64 ** -0.5)
    assert_rounded(out.view(want.shape), want, F16, bound[..., None])
    # lengths past max_len are cut and reported
    Q.stagq_kv_attention(c.cache, q, c.table, c.lens, out, max_len=16)
    with pytest.raises(Q.StagqError):
        Q.stagq_ops_check(0)
    want, _, bound, _ = R.attention(q.cpu().view(2, 1, 4, 64), c.k, c.v, [16, 16], 1, 64 ** -0.5)
    assert_rounded(out.view(want.shape), want, F16, bound[..., None])


@gpu
@pytest.mark.parametrize("dim,group,page,dtype", FORMATS)
@pytest.mark.parametrize("q_heads,n_new", [(2, 1), (8, 1), (4, 3), (14, 2), (16, 5)])
def test_attention_against_64_bits(dim, group, page, dtype, q_heads, n_new):
    # one token, an end inside a page and a tile, an empty sequence, fewer tokens than queries, many tiles
    c = Case([1, 31, 0, 2, 33, 128, 517], 2, dim, page, group, dtype)
    c.check(q_heads, n_new)
    c.check(q_heads, n_new, tracked=True)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_over_a_long_sequence_split_over_the_gpu(dtype):
    c = Case([4500], 1, 128, 64, 64, dtype)
    c.check(4, 1)
    c.check(4, 2, tracked=True)


@gpu
def test_attention_scales_of_very_different_size():
    # groups of V whose scales are 2^24 apart and in either order, and scores with one large peak
    v = rnd((1, 300, 2, 128), 4, BF16)
    v[0, :100] *= 2.0 ** -30
    v[0, 200:, :, :64] *= 2.0 ** 20
    k = rnd((1, 300, 2, 128), 5, BF16)
    k[0, 250] *= 9
    Case([300], 2, 128, 16, 64, BF16, v=v, k=k).check(8, 1)
    Case([300], 2, 128, 16, 64, BF16, v=v.flip(1), k=k).check(8, 2, tracked=True)
    Case([300], 2, 128, 16, 64, BF16, v=(v.double() * 2.0 ** -100).to(BF16), k=k).check(8, 1)
    Case([70], 2, 64, 16, 64, F16, v=rnd((1, 70, 2, 64), 6, F16, 1e-6)).check(4, 1)
    # q far from 1, and other softmax scales
    c = Case([90], 2, 128, 16, 128, BF16)
    q = rnd((1, 4 * 128), 8, BF16)
    c.check(4, 1, q=(q.double() * 2.0 ** 60).to(BF16), scale=2.0 ** -64)
    c.check(4, 1, q=(q.double() * 2.0 ** -60).to(BF16), scale=2.0 ** 56)
    c.check(4, 1, scale=-0.3)
    c.check(4, 1, scale=0.0)


@gpu
def test_attention_keeps_what_a_row_may_not_see_out():
    # NaN and infinity in a token that only the last of three queries sees, in K of one head and V of the other
    k, v = rnd((1, 40, 2, 128), 1, F16), rnd((1, 40, 2, 128), 2, F16)
    k[0, 39, 0, 3], v[0, 39, 1, 100] = float("nan"), float("inf")
    c = Case([40], 2, 128, 16, 64, F16, k=k, v=v)
    q = rnd((3, 4 * 128), 3, F16).cuda()
    mass = torch.zeros(1, 2, c.width * 16, device="cuda")
    out = c.attend(q, 3, mass).view(3, 2, 2, 128).cpu()
    clean_k, clean_v = c.k.clone(), c.v.clone()
    clean_k[0, 39], clean_v[0, 39] = 0, 0
    want, _, bound, _ = R.attention(q.cpu().view(1, 3, 4, 128), clean_k, clean_v, [40], 3, 128 ** -0.5)
    assert_rounded(out[:2].flatten(1, 2), want[0, :2], F16, bound[0, :2, :, None])
    assert torch.isnan(out[2, 0]).all()                                  # K: every weight of that head's last query
    assert torch.isnan(out[2, 1, :, 64:]).all() and torch.isfinite(out[2, 1, :, :64]).all()  # V: its group alone
    assert torch.isnan(mass[0, 0, :40]).all() and torch.isfinite(mass[0, 1]).all() and not mass[0, :, 40:].any()


@gpu
def test_attention_takes_slices_other_streams_and_workspaces():
    c = Case([700, 45], 2, 128, 32, 128, F16)
    qkv = rnd((2, 3 + 8 * 128 + 5), 3, F16).cuda()
    q = qkv[:, 3:3 + 8 * 128]                                           # rows not on 16 bytes
    want = c.check(8, 1, q=q.cpu().contiguous())
    whole = torch.full((2, 2000), 3.0, dtype=F16, device="cuda")
    need = Q.stagq_kv_attention_workspace(c.cache, 2, c.width * 32, 8, tracked=True)
    mass = torch.zeros(2, 2, c.width * 32, device="cuda")
    with pytest.raises(Q.StagqError):
        Q.stagq_kv_attention(c.cache, q, c.table, c.lens, whole[:, 5:1029], mass=mass, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Q.stagq_kv_attention(c.cache, q, c.table, c.lens, whole[:, 5:1029], stream=s)
    s.synchronize()
    assert torch.equal(whole[:, 5:1029], want)
    whole.fill_(3.0)
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    Q.stagq_kv_attention(c.cache, q, c.table, c.lens, whole[:, 5:1029], mass=mass, workspace=ws, stream=s)
    s.synchronize()
    out, _, bound, _ = R.attention(q.cpu().reshape(2, 1, 8, 128), c.k, c.v, c.lens_l, 1, 128 ** -0.5)
    assert_rounded(whole[:, 5:1029].reshape(out.shape), out, F16, bound[..., None])
    want = whole[:, 5:1029].clone()
    s.synchronize()
    assert torch.equal(whole[:, 5:1029], want)
    assert (whole[:, :5] == 3).all() and (whole[:, 1029:] == 3).all()
    for _ in range(3):  # the same bits every time, mass included
        m = [torch.zeros(2, 2, c.width * 32, device="cuda") for _ in range(2)]
        assert torch.equal(c.attend(q, 1, m[0]), c.attend(q, 1, m[1])) and torch.equal(m[0], m[1])
    padded = torch.zeros(2, 2, 2000, device="cuda")[:, :, :c.width * 32]  # mass rows further apart
    c.attend(q, 1, padded)
    assert torch.equal(padded, m[0])


@gpu
def test_captured_decode_step_follows_growing_lengths():
    # append and attention in one graph; starts and lens change between replays
    c = Case([30, 7], 2, 128, 16, 128, F16, width=8)
    n = c.width * 16
    starts, lens = c.lens.clone(), c.lens + 1
    q, k, v = (torch.empty(2, w * 128, dtype=F16, device="cuda") for w in (8, 2, 2))
    out, mass = torch.empty(2, 8 * 128, dtype=F16, device="cuda"), torch.zeros(2, 2, n, device="cuda")
    ws = torch.empty(Q.stagq_kv_attention_workspace(c.cache, 2, n, 8, tracked=True), dtype=torch.uint8, device="cuda")

    def step():
        Q.stagq_kv_append(c.cache, k, v, c.table, starts, 1)
        Q.stagq_kv_attention(c.cache, q, c.table, lens, out, mass=mass, workspace=ws)

    ks, vs = [list(c.k[i, :m]) for i, m in enumerate((30, 7))], [list(c.v[i, :m]) for i, m in enumerate((30, 7))]
    q.zero_(), k.zero_(), v.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    mass.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    total, slack = torch.zeros(2, 2, n, dtype=torch.float64), torch.zeros(2, 2, n, dtype=torch.float64)
    for i in range(20):
        new = [rnd((2, w * 128), 50 + 3 * i + w, F16) for w in (8, 2, 2)]
        new[2] = rnd((2, 2 * 128), 900 + i, F16)
        for dst, x in zip((q, k, v), new):
            dst.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        for b in range(2):
            ks[b].append(R.values4(new[1][b].view(2, 128), 128))
            vs[b].append(R.values4(new[2][b].view(2, 128), 128))
            kk, vv = torch.stack(ks[b])[None], torch.stack(vs[b])[None]
            want, p, bound, p_bound = R.attention(new[0][b].view(1, 1, 8, 128), kk, vv, [len(ks[b])], 1, 128 ** -0.5)
            assert_rounded(out[b].view(want.shape), want, F16, bound[..., None], f"step {i}")
            total[b, :, :len(ks[b])] += p[0]
            slack[b, :, :len(ks[b])] += p_bound[0] + 2.0 ** -24 * total[b, :, :len(ks[b])]
        starts += 1
        lens += 1
    assert ((mass.double().cpu() - total).abs() <= slack * (1 + 2.0 ** -20)).all()
    Q.stagq_ops_check(0)


@gpu
@pytest.mark.parametrize("lens", [[0], [1], [130], [700, 0, 33], [0, 0, 0, 0, 5000]])
def test_attention_of_short_sequences_under_a_large_capacity(lens):
    # the work is laid out for max_len: most CTAs have none, and a workspace of
    # junk and page numbers past a sequence's last page are never read
    b, heads, dim, page, width = len(lens), 2, 128, 64, 4096
    c = Case(lens, heads, dim, page, 128, F16)
    table = torch.full((b, width), -7, dtype=torch.int32, device="cuda")
    table[:, :c.width] = c.table
    q = rnd((2 * b, 8 * dim), 3, F16)
    want, p, bound, p_bound = R.attention(q.view(b, 2, 8, dim), c.k, c.v, lens, 2, dim ** -0.5)
    for max_len in (width * page, max(max(lens), 1)):
        for tracked in (False, True):
            mass = torch.zeros(b, heads, width * page, device="cuda") if tracked else None
            need = Q.stagq_kv_attention_workspace(c.cache, b, max_len, 8, 2, tracked)
            ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
            out = torch.full((2 * b, 8 * dim), 3.0, dtype=F16, device="cuda")
            for _ in range(2):  # and a workspace that holds the last call's sums
                Q.stagq_kv_attention(c.cache, q.cuda(), table, c.lens, out, n_new=2, mass=mass, max_len=max_len, workspace=ws)
                Q.stagq_ops_check(0)
                assert_rounded(out.view(want.shape), want, F16, bound[..., None], f"{max_len} {tracked}")
            assert (ws[need:] == 0xFF).all()
            if tracked:
                n = p.shape[2]
                assert ((mass[:, :, :n].double().cpu() - 2 * p).abs() <= 2 * p_bound + 2.0 ** -22 * p).all()
                assert not mass[:, :, n:].any()


@gpu
def test_calls_on_two_streams_at_once():
    c = Case([900, 31], 2, 128, 32, 64, BF16)
    jobs = []
    for i in range(2):
        a, xs, b, ws, _ = _i8(300, 2048, 700, 40 + i)
        x = rnd((300, 2048), 60 + i, BF16).cuda()
        q = rnd((2, 8 * 128), 50 + i, BF16).cuda()

        def job(x=x, b=b, ws=ws, q=q, stream=None):
            n, w = x.shape[0], b.shape[1]
            xq, xs = torch.empty(n, w, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
            y, small = torch.empty(n, 700, device="cuda"), torch.empty(9, 700, device="cuda")
            out, mass = torch.empty_like(q), torch.zeros(2, 2, c.width * 32, device="cuda")
            Q.stagq_quantize_i8(x, xq, xs)
            Q.stagq_gemm_i8(xq, xs, b, ws, 2048, y)
            Q.stagq_gemm_i8(xq[:9], xs[:9], b, ws, 2048, small)
            Q.stagq_kv_attention(c.cache, q, c.table, c.lens, out, mass=mass)
            return y, small, out, mass

        jobs.append((job, [t.clone() for t in job()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for job, _, stream in jobs:
            with torch.cuda.stream(stream):
                got.append(job())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for have, want in zip(outs, jobs[i % 2][1]):
            assert torch.equal(have, want), i
    Q.stagq_ops_check(0)


@gpu
def test_attention_reads_offsets_beyond_32_bits():
    # a pool of more than 4 GiB whose used pages lie at its end
    heads, dim, page = 8, 128, 64
    size = Q.stagq_kv_page_bytes(heads, dim, page, 128)
    n_pages = (1 << 32) // size + 8
    pool = torch.empty(n_pages, size, dtype=torch.uint8, device="cuda")
    cache = Q.KVCache(pool, heads, dim, page, 128, F16)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 3]], dtype=torch.int32, device="cuda")
    k, v, q = (rnd((r, w * dim), s, F16) for r, w, s in ((150, heads, 1), (150, heads, 2), (1, 32, 3)))
    Q.stagq_kv_append(cache, k.cuda(), v.cuda(), table, torch.zeros(1, dtype=torch.int32, device="cuda"), 150)
    out = torch.empty(1, 32 * dim, dtype=F16, device="cuda")
    Q.stagq_kv_attention(cache, q.cuda(), table, torch.tensor([150], dtype=torch.int32, device="cuda"), out)
    kk, vv = (R.values4(x.view(1, 150, heads, dim), 128) for x in (k, v))
    want, _, bound, _ = R.attention(q.view(1, 1, 32, dim), kk, vv, [150], 1, dim ** -0.5)
    assert_rounded(out.view(want.shape), want, F16, bound[..., None])
    Q.stagq_ops_check(0)


# ------------------------------------------------------------------------ eviction

@gpu
@pytest.mark.parametrize("dim,group,page,dtype", FORMATS)
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (20, 5), (33, 33), (64, 0), (100, 7)])
def test_evict_keeps_the_largest_masses(dim, group, page, dtype, budget, recent):
    lens, heads = [1, 20, 97, 300], 2
    c = Case(lens, heads, dim, page, group, dtype, spare=4 * -(-budget // page))
    before = c.pool.clone()
    fresh = c.unused.reshape(4, -1).cuda()
    mass = torch.floor(torch.rand(4, heads, c.width * page, generator=torch.Generator().manual_seed(1)) * 8)  # many ties
    mass[3, 0, :300] = torch.randn(300, generator=torch.Generator().manual_seed(2))                            # negative ones
    mass[3, 1, 5], mass[3, 1, 9], mass[3, 1, 11], mass[2, 1, 3], mass[2, 1, 4] = float("nan"), float("inf"), float("-inf"), -0.0, 0.0
    cap = budget + 3
    kept = torch.empty(4, heads, budget, dtype=torch.int32, device="cuda")
    new_lens, new_mass = torch.empty(4, dtype=torch.int32, device="cuda"), torch.full((4, heads, cap), 5.0, device="cuda")
    Q.stagq_kv_evict(c.cache, c.table, c.lens, mass.cuda(), fresh, budget, recent, kept, new_lens, new_mass)
    Q.stagq_ops_check(0)
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    k, v = (torch.empty(4 * budget, heads * dim, device="cuda") for _ in range(2))
    Q.stagq_kv_read(c.cache, fresh, new_lens, k, v, budget)
    k, v = (x.view(4, budget, heads, dim) for x in (k, v))
    for b, n in enumerate(lens):
        for h in range(heads):
            want = R.keep(mass[b, h].numpy(), n, budget, recent)
            m = len(want)
            assert kept[b, h].tolist() == want + [-1] * (budget - m), (b, h)
            assert torch.equal(new_mass[b, h, :m].cpu().nan_to_num(7.5), mass[b, h, want].nan_to_num(7.5))
            assert not new_mass[b, h, m:].any()
            assert_rounded(k[b, :m, h], c.k[b, want, h], F32)
            assert_rounded(v[b, :m, h], c.v[b, want, h], F32)
    old = c.table.flatten().long()
    assert torch.equal(c.pool[old], before[old])  # the old pages are only read


@gpu
def test_evict_on_equal_and_long_masses():
    n = 5000
    c = Case([n], 1, 64, 64, 64, F16, spare=16)
    fresh = c.unused[:16].reshape(1, 16).cuda()
    kept = torch.empty(1, 1, 1024, dtype=torch.int32, device="cuda")
    new_lens, new_mass = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, 1, 1024, device="cuda")
    for mass in (torch.zeros(1, 1, 5056), torch.rand(1, 1, 5056, generator=torch.Generator().manual_seed(3)) * 1e-6,
                 torch.arange(5056.).view(1, 1, -1) % 7):
        Q.stagq_kv_evict(c.cache, c.table, c.lens, mass.cuda(), fresh, 1024, 100, kept, new_lens, new_mass)
        assert kept[0, 0].tolist() == R.keep(mass[0, 0].numpy(), n, 1024, 100)
    Q.stagq_ops_check(0)


@gpu
@pytest.mark.parametrize("lens,budget,recent", [([70000, 3, 900], 900, 33), ([33000], 20000, 0), ([300000], 700, 700), ([300000], 1000, 17)])
def test_evict_of_long_sequences(lens, budget, recent):
    # selections shared by several CTAs, one sequence that is copied whole among them, and one too long for the registers
    b, page, heads = len(lens), 1024, 2
    per, fresh_per = -(-max(lens) // page), -(-budget // page)
    size = Q.stagq_kv_page_bytes(heads, 64, page, 64)
    pool = torch.randint(0, 60, (b * (per + fresh_per), size), dtype=torch.uint8, device="cuda")
    cache = Q.KVCache(pool, heads, 64, page, 64, F16)
    order = torch.randperm(b * (per + fresh_per), generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    table, fresh = order[:b * per].view(b, per), order[b * per:].view(b, fresh_per)
    mass = torch.rand(b, heads, per * page, generator=torch.Generator().manual_seed(5))
    mass[:, 1] = torch.floor(mass[:, 1] * 50)  # ties across the CTAs' slices
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept, new_lens = torch.empty(b, heads, budget, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
    new_mass = torch.empty(b, heads, budget, device="cuda")
    Q.stagq_kv_evict(cache, table, n, mass.cuda(), fresh, budget, recent, kept, new_lens, new_mass)
    Q.stagq_ops_check(0)
    rows = max(lens)
    old_k, old_v = (torch.empty(b * rows, heads * 64, device="cuda") for _ in range(2))
    Q.stagq_kv_read(cache, table, n, old_k, old_v, rows)
    k, v = (torch.empty(b * budget, heads * 64, device="cuda") for _ in range(2))
    Q.stagq_kv_read(cache, fresh, new_lens, k, v, budget)
    for i in range(b):
        for h in range(heads):
            want = R.keep(mass[i, h].numpy(), lens[i], budget, recent)
            assert kept[i, h].tolist() == want + [-1] * (budget - len(want))
            at = torch.tensor(want, device="cuda")
            for new, old in ((k, old_k), (v, old_v)):
                assert torch.equal(new.view(b, budget, heads, 64)[i, :len(want), h], old.view(b, rows, heads, 64)[i, at, h])
            assert torch.equal(new_mass[i, h, :len(want)].cpu(), mass[i, h, want])


@gpu
def test_kv_binding_refuses_what_does_not_fit():
    c = Case([20, 20], 2, 64, 16, 64, F16)
    k = torch.zeros(2, 128, dtype=F16, device="cuda")
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 256, dtype=F16, device="cuda")
    for bad in (dict(k=k[:1]), dict(v=k[:, :64]), dict(table=c.table[:1]), dict(starts=z[:1]), dict(starts=z.cpu()), dict(table=c.table.t())):
        a = {**dict(k=k, v=k, table=c.table, starts=z), **bad}
        with pytest.raises(ValueError):
            Q.stagq_kv_append(c.cache, a["k"], a["v"], a["table"], a["starts"], 1)
    for bad in (dict(k=k.to(BF16)), dict(starts=z.long()), dict(table=c.table.long())):
        a = {**dict(k=k, v=k, table=c.table, starts=z), **bad}
        with pytest.raises(TypeError):
            Q.stagq_kv_append(c.cache, a["k"], a["v"], a["table"], a["starts"], 1)
    mass = torch.zeros(2, 2, 32, device="cuda")
    for bad in (dict(q=q[:, :200]), dict(out=q[:1]), dict(lens=z[:1]), dict(mass=mass[:1]), dict(mass=mass[:, :1]), dict(max_len=33),
                dict(workspace=torch.zeros(8, dtype=torch.uint8))):
        a = {**dict(q=q, table=c.table, lens=c.lens, out=q), **bad}
        with pytest.raises(ValueError):
            Q.stagq_kv_attention(c.cache, **a)
    three = Q.KVCache(torch.zeros(Q.stagq_kv_page_bytes(3, 64, 16, 64), dtype=torch.uint8, device="cuda"), 3, 64, 16, 64, F16)
    with pytest.raises(ValueError):  # 4 query heads are no multiple of 3 KV heads
        Q.stagq_kv_attention(three, q, c.table, c.lens, q.clone())


# ------------------------------------------------------------------ run together

@gpu
def test_a_layers_prompt_decode_and_eviction():
    """One attention layer as a served model runs it: the prompt through the
    8-bit linears, its K and V into the cache, then decode steps with the StagQ
    GEMV for q/k/v and o, then an eviction and one more step."""
    d, heads, qh, dim, group = 512, 2, 8, 64, 64
    sizes = [qh * dim, heads * dim, heads * dim]
    W = [synth.weights(s, d, seed=20 + i) for i, s in enumerate(sizes)]
    Wo = synth.weights(d, qh * dim, seed=30)
    qkv = Q.stagq_load_stack([Q.stagq_pack(Q.stagq_encode(w, 128, 2, 0.005, "fast")) for w in W], 0)
    o = Q.stagq_load(Q.stagq_pack(Q.stagq_encode(Wo, 128, 2, 0.005, "fast")), 0)
    from oracle import stagq as O
    enc = [O.encode(w, 128, 2, 0.005, "fast") for w in W]
    enc_o = O.encode(Wo, 128, 2, 0.005, "fast")

    # prompt: K and V of 50 tokens by the 8-bit linear on the stacked weights
    n, page, width = 50, 16, 8
    w = torch.from_numpy(np.concatenate(W)).cuda()
    wq, ws = torch.empty(w.shape[0], 512, dtype=torch.int8, device="cuda"), torch.empty(w.shape[0], device="cuda")
    Q.stagq_quantize_i8(w, wq, ws)
    x = torch.from_numpy(synth.activations(n, d, 1)).cuda()
    xq, xs = torch.empty(n, 512, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    Q.stagq_quantize_i8(x, xq, xs)
    y = torch.empty(n, sum(sizes), dtype=F16, device="cuda")
    Q.stagq_gemm_i8(xq, xs, wq, ws, d, y)
    a, sa = R.quantize_i8(x.cpu())
    b, sb = R.quantize_i8(w.cpu())
    want_y = (a @ b.T) * sa[:, None] * sb
    assert_rounded(y, want_y, F16, want_y.abs() * 5.01 * 2.0 ** -24)  # 3 roundings, and one in each scale

    pool = torch.zeros(2 * width, Q.stagq_kv_page_bytes(heads, dim, page, group), dtype=torch.uint8, device="cuda")
    cache = Q.KVCache(pool, heads, dim, page, group, F16)
    table = torch.randperm(2 * width, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(2, 1, width).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    Q.stagq_kv_append(cache, y[:, sizes[0]:sizes[0] + sizes[1]], y[:, sizes[0] + sizes[1]:], table[0], lens - n, n)
    k, v = (R.values4(t.reshape(n, heads, dim).cpu(), group) for t in y[:, sizes[0]:].split(sizes[1:], 1))
    mass, live = torch.zeros(1, heads, width * page, device="cuda"), table[0]

    def decode(i, k, v):
        xi = synth.activations(1, d, 100 + i)
        yi = torch.empty(1, sum(sizes), dtype=F16, device="cuda")
        Q.stagq_gemv(qkv, 4, torch.from_numpy(xi).cuda(), yi)
        ref = np.concatenate([O.gemv(e, 4, xi)[0] for e in enc])
        assert np.linalg.norm(yi.float().cpu().numpy()[0] - ref) <= 1e-3 * np.linalg.norm(ref)
        starts = lens.clone()
        lens.add_(1)
        Q.stagq_kv_append(cache, yi[:, sizes[0]:sizes[0] + sizes[1]], yi[:, sizes[0] + sizes[1]:], live, starts, 1)
        at, mass_before = torch.empty(1, qh * dim, dtype=F16, device="cuda"), mass[0].clone()
        Q.stagq_kv_attention(cache, yi[:, :sizes[0]], live, lens, at, mass=mass)
        nk, nv = (R.values4(t.reshape(1, heads, dim).cpu(), group) for t in yi[:, sizes[0]:].split(sizes[1:], 1))
        k, v = torch.cat([k, nk]), torch.cat([v, nv])
        out, p, bound, p_bound = R.attention(yi[:, :sizes[0]].cpu().view(1, 1, qh, dim), k[None], v[None], [k.shape[0]], 1, dim ** -0.5)
        assert_rounded(at.view(out.shape), out, F16, bound[..., None], f"step {i}")
        z = torch.empty(1, d, dtype=F16, device="cuda")
        Q.stagq_gemv(o, 4, at, z)
        ref = O.gemv(enc_o, 4, at.cpu().numpy())[0]
        assert np.linalg.norm(z.float().cpu().numpy()[0] - ref) <= 1e-3 * np.linalg.norm(ref)
        old, m = mass_before.double().cpu(), k.shape[0]
        assert ((mass[0, :, :m].double().cpu() - old[:, :m] - p[0, :, :m]).abs() <= p_bound[0, :, :m] + 2.0 ** -24 * (old[:, :m] + p[0, :, :m])).all()
        return k, v

    for i in range(4):
        k, v = decode(i, k, v)
    kept = torch.empty(1, heads, 24, dtype=torch.int32, device="cuda")
    new_lens, new_mass = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, heads, width * page, device="cuda")
    Q.stagq_kv_evict(cache, live, lens, mass, table[1], 24, 6, kept, new_lens, new_mass)
    idx = [R.keep(mass[0, h].cpu().numpy(), 54, 24, 6) for h in range(heads)]
    assert kept[0].tolist() == idx
    k, v = (torch.stack([t[idx[h], h] for h in range(heads)], 1) for t in (k, v))
    lens, live, mass = new_lens, table[1], new_mass
    decode(9, k, v)
    assert lens.tolist() == [25]
    Q.stagq_ops_check(0)
