"""bf16 grouped products against their 64-bit forms.

Sums are in fp32: of k terms with total size s = sum |a| |b| each of the at most k additions loses 2^-23 of s (whether it
rounds or truncates), and the output is rounded once, by half a step (bf16 2^-8, fp32 2^-24).  On small
integers every sum is exact, and the outputs are the rounded exact values."""
import pytest
import torch

import fp8_moe_expert_gb300 as fme
from tests import block128 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    fme.ensure_built()


@pytest.fixture(autouse=True)
def _nothing_cached():
    """No memory but the test's own is mapped: an access next to a tensor has less to hit."""
    torch.cuda.empty_cache()


@pytest.fixture
def status():
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    yield st
    assert fme.read_device_status(st)[0] == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def integers(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(torch.bfloat16)


def near(y, want, size, terms):
    err = (y.double() - want).abs()
    allowed = HALF[y.dtype] * want.abs() + (terms + 1) * 2.0 ** -23 * size
    assert bool((err <= allowed).all()), float((err - allowed).max())


def forward64(x, w, off):
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(y)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = x[lo:hi].double(), w[e].double().t()
        y[lo:hi], size[lo:hi] = a @ b, a.abs() @ b.abs()
    return y, size


# rows, experts, n, k: those of the first three lines are in the form for few rows, the others in tiles
FORWARD = [(1, 1, 8, 8), (1, 4, 128, 64), (3, 2, 136, 72), (16, 1, 256, 200), (17, 3, 1048, 1400), (64, 1, 129 * 8, 512),
           (65, 1, 256, 64), (200, 40, 384, 328), (288, 1, 64, 64), (289, 1, 64, 64), (600, 2, 8, 16), (700, 3, 264, 24),
           (1500, 5, 520, 72), (4000, 7, 256, 512), (33100, 1024, 40, 136),
           (1999, 8, 1048, 1400), (9000, 5, 520, 72), (9000, 7, 256, 512), (10000, 2, 8, 16), (15000, 1, 72, 8),
           (60000, 1024, 40, 136)]


@pytest.mark.parametrize("rows,experts,n,k", FORWARD)
def test_forward(rows, experts, n, k, status):
    off = ref.split(rows, experts, rows + n)
    x, w = ref.normal((rows, k), 1.0, 1), ref.normal((experts, n, k), 0.05, 2)
    y = fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=status)
    near(y, *forward64(x, w, off), k)
    x, w = integers((rows, k), 3), integers((experts, n, k), 4)
    y = fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=status)
    assert torch.equal(y, forward64(x, w, off)[0].to(torch.bfloat16))


DGRAD = [(1, 1, 8, 8), (5, 3, 128, 256), (130, 4, 136, 264), (257, 1, 64, 520), (1999, 8, 1048, 1400), (700, 200, 72, 40)]


@pytest.mark.parametrize("rows,experts,n,k", DGRAD)
def test_dgrad(rows, experts, n, k, status):
    off = ref.split(rows, experts, rows + n)
    for make, exact in ((lambda s, i: ref.normal(s, 0.5, i), False), (integers, True)):
        dy, w = make((rows, n), 1), make((experts, n, k), 2)
        dx = fme.grouped_gemm_dgrad_bf16(dy, w, i32(off), status=status)
        want, size = forward64(dy, w.transpose(1, 2), off)
        near(dx, want, size, n)
        if exact:
            assert torch.equal(dx, want.to(torch.bfloat16))


def wgrad64(dy, x, off):
    e = len(off) - 1
    dw = torch.zeros((e, dy.shape[1], x.shape[1]), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(dw)
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        a, b = dy[lo:hi].double().t(), x[lo:hi].double()
        dw[i], size[i] = a @ b, a.abs() @ b.abs()
    return dw, size


WGRAD = [(0, 3, 64, 64), (1, 1, 8, 8), (63, 1, 72, 128), (64, 1, 128, 256), (65, 2, 136, 264), (200, 5, 264, 72),
         (1999, 8, 1048, 1400), (700, 200, 72, 40), (5000, 3, 256, 520)]


@pytest.mark.parametrize("rows,experts,n,k", WGRAD)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad(rows, experts, n, k, dtype, status):
    off = ref.split(rows, experts, rows + n)
    for make, exact in ((lambda s, i: ref.normal(s, 0.5, i), False), (integers, True)):
        dy, x = make((rows, n), 1), make((rows, k), 2)
        dw = fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dtype=dtype, status=status)
        assert dw.dtype == dtype
        want, size = wgrad64(dy, x, off)
        near(dw, want, size, rows)
        if exact:
            assert torch.equal(dw, want.to(dtype))


@pytest.mark.parametrize("rows,experts,n,k", WGRAD)
def test_wgrad_added_into_fp32(rows, experts, n, k, status):
    off = ref.split(rows, experts, rows + n)
    dy, x = ref.normal((rows, n), 0.5, 1), ref.normal((rows, k), 0.5, 2)
    acc = torch.randn((experts, n, k), device=DEV)
    want = acc + fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dtype=torch.float32, status=status)
    out = fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dw=acc, accumulate=True, status=status)
    assert out is acc and torch.equal(acc, want)


def test_long_wgrad_in_fp32_is_rounded_block_by_block(status):
    """The sums of 1024 rows are exact here (products below 2^14), so the result is theirs, added in order in fp32."""
    off, n, k = [0, 20000, 20037, 21061, 46661], 264, 136
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    dy, x = (torch.randint(0, 128, (off[-1], c), generator=g, device=DEV).to(torch.bfloat16) for c in (n, k))
    want = torch.zeros((4, n, k), device=DEV)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        for at in range(lo, hi, 1024):
            to = min(at + 1024, hi)
            want[e] += (dy[at:to].double().t() @ x[at:to].double()).float()
    assert torch.equal(fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dtype=torch.float32, status=status), want)
    old = torch.randn((4, n, k), device=DEV) * 1e6
    out = fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), dw=old.clone(), accumulate=True, status=status)
    assert torch.equal(out, old + want)


def test_a_rows_bits_do_not_depend_on_the_batch(status):
    """One row alone, a few (the form for few rows) and the whole batch (tiles)."""
    rows, experts, n, k = 6000, 3, 392, 1352
    off = [0, 500, 500, 6000]
    x, w = ref.normal((rows, k), 1.0, 1), ref.normal((experts, n, k), 0.05, 2)
    y = fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=status)
    few = fme.grouped_gemm_fwd_bf16(x[450:600].contiguous(), w, i32([0, 50, 50, 150]), status=status)
    assert torch.equal(few, y[450:600])
    for r in (0, 499, 500, 899, 5999):
        e = 0 if r < 500 else 2
        one = fme.grouped_gemm_fwd_bf16(x[r:r + 1], w, i32([0] * (e + 1) + [1] * (experts - e)), status=status)
        assert torch.equal(one[0], y[r])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("off", [[0, 70, 70, 133, 300], [0, 70, 70, 133, 9000]])
def test_one_experts_values_do_not_reach_anothers(off, bad, status):
    rows, n, k = off[-1], 136, 200
    dy, x, w = ref.normal((rows, n), 0.5, 1), ref.normal((rows, k), 0.5, 2), ref.normal((4, n, k), 0.05, 3)
    clean = (fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), status=status),
             fme.grouped_gemm_dgrad_bf16(dy, w, i32(off), status=status),
             fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=status))
    for t in (dy, x):
        t[off[2]:off[3]] = bad
    w[1] = bad  # the expert without rows
    w[2] = bad
    dw = fme.grouped_gemm_wgrad_bf16(dy, x, i32(off), status=status)
    assert torch.equal(dw[[0, 1, 3]], clean[0][[0, 1, 3]]) and not bool(dw[2].isfinite().any())
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[off[2]:off[3]] = False
    for got, want in ((fme.grouped_gemm_dgrad_bf16(dy, w, i32(off), status=status), clean[1]),
                      (fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=status), clean[2])):
        assert torch.equal(got[keep], want[keep]) and not bool(got[~keep].isfinite().any())


@pytest.mark.parametrize("n", [40, 1000, 4096, 9000])
@pytest.mark.parametrize("k", [64, 200, 520, 1400])
def test_forward_of_few_rows_in_items_of_any_height(n, k, status):
    """Items of 32, 64 and 128 rows of W, with blocks of 64 of k that do not fill a stage; a NaN row of W stays its own."""
    for rows, experts in ((1, 1), (16, 1), (3, 5), (17, 1), (32, 2), (33, 1)):
        off = ref.split(rows, experts, rows + n)
        x, w = integers((rows, k), 1), integers((experts, n, k), 2)
        w[:, 33 % n] = float("nan")
        y = fme.grouped_gemm_fwd_bf16(x, w, i32(off), status=status)
        want, _ = forward64(x, w, off)
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(), want.to(torch.bfloat16).nan_to_num())


@pytest.mark.parametrize("n,k", [(128, 320), (136, 200), (1088, 72)])
def test_wgrad_ends_anywhere(n, k, status):
    """Ends within the first 64 rows, each distance from a step of 16 and from a block of 64, NaN in every other expert's rows."""
    sizes = [3, 13, 16, 15, 0, 17, 1, 47, 64, 63, 65, 1, 128, 79, 80, 81, 127, 200] + [64 + 3 * i for i in range(22)]
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    dy, x = integers((off[-1], n), 1), integers((off[-1], k), 2)
    want = wgrad64(dy, x, off)[0].to(torch.float32)
    for odd in (0, 1):
        a, b = dy.clone(), x.clone()
        for e in range(odd, len(sizes), 2):
            a[off[e]:off[e + 1]], b[off[e]:off[e + 1]] = float("nan"), float("inf")
        dw = fme.grouped_gemm_wgrad_bf16(a, b, i32(off), dtype=torch.float32, status=status)
        assert torch.equal(dw[1 - odd::2], want[1 - odd::2])
        full = [e for e in range(odd, len(sizes), 2) if sizes[e]]
        assert not bool(dw[full].isfinite().any())


@pytest.mark.parametrize("offsets", [[0, 5, 3, 300], [1, 5, 9, 300], [0, 5, 9, 299], [0, 5, 9, 301], [0, -5, 9, 300]])
def test_malformed_offsets_are_reported_and_nothing_is_written(offsets):
    rows, n, k = 30000, 64, 72
    dy, x, w = ref.normal((rows, n), 0.5, 1), ref.normal((rows, k), 0.5, 2), ref.normal((3, n, k), 0.05, 3)
    for m in (rows, 40):  # in tiles, and the form for few rows
        off = i32([o if o < 299 else o - 300 + m for o in offsets])
        for call, out in ((lambda st, o: fme.grouped_gemm_fwd_bf16(x[:m], w, off, y=o, status=st), (m, n)),
                          (lambda st, o: fme.grouped_gemm_dgrad_bf16(dy[:m], w, off, dx=o, status=st), (m, k)),
                          (lambda st, o: fme.grouped_gemm_wgrad_bf16(dy[:m], x[:m], off, dw=o, status=st), (3, n, k))):
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            o = torch.full(out, 7.0, dtype=torch.bfloat16, device=DEV)
            call(st, o)
            assert fme.read_device_status(st)[0] == fme.ERR_DEVICE_BAD_OFFSETS
            assert bool((o == 7.0).all())


@pytest.mark.parametrize("rows", [333, 3333])
def test_nothing_outside_the_outputs_is_written(rows, status):
    experts, n, k = 4, 1048, 88
    off = i32(ref.split(rows, experts, 5))
    dy, x, w = ref.normal((rows, n), 0.5, 1), ref.normal((rows, k), 0.5, 2), ref.normal((experts, n, k), 0.05, 3)

    def banded(shape, dtype):
        count = 1
        for d in shape:
            count *= d
        whole = torch.full((count + 2048,), 7.0, dtype=dtype, device=DEV)
        return whole, whole[1024:1024 + count].view(shape)

    for shape, dtype, call in (
            ((rows, n), torch.bfloat16, lambda o: fme.grouped_gemm_fwd_bf16(x, w, off, y=o, status=status)),
            ((40, n), torch.bfloat16, lambda o: fme.grouped_gemm_fwd_bf16(x[:40], w, i32([0, 3, 3, 40, 40]), y=o,
                                                                          status=status)),
            ((rows, k), torch.bfloat16, lambda o: fme.grouped_gemm_dgrad_bf16(dy, w, off, dx=o, status=status)),
            ((experts, n, k), torch.bfloat16, lambda o: fme.grouped_gemm_wgrad_bf16(dy, x, off, dw=o, status=status)),
            ((experts, n, k), torch.float32, lambda o: fme.grouped_gemm_wgrad_bf16(dy, x, off, dw=o, status=status))):
        whole, out = banded(shape, dtype)
        call(out)
        assert bool((whole[:1024] == 7.0).all()) and bool((whole[-1024:] == 7.0).all())


def test_captured_and_replayed_with_other_loads(status):
    """A graph of the three products, replayed after the rows and their grouping changed."""
    rows, experts, n, k = 9000, 4, 136, 264
    dy, x, w = ref.normal((rows, n), 0.5, 1), ref.normal((rows, k), 0.5, 2), ref.normal((experts, n, k), 0.05, 3)
    off = i32([0, 100, 350, 350, 9000])

    def calls():
        return (fme.grouped_gemm_fwd_bf16(x, w, off, status=status), fme.grouped_gemm_dgrad_bf16(dy, w, off, status=status),
                fme.grouped_gemm_wgrad_bf16(dy, x, off, status=status))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    x.copy_(ref.normal((rows, k), 0.5, 7))
    off.copy_(i32([0, 0, 1, 8990, 9000]))
    for _ in range(2):
        for o in out:
            o.fill_(0)
        graph.replay()
        for got, want in zip(out, calls()):
            assert torch.equal(got, want)


def test_on_a_stream_of_its_own(status):
    rows, experts, n, k = 9000, 3, 264, 520
    off = i32([0, 120, 120, 9000])
    dy, x, w = ref.normal((rows, n), 0.5, 1), ref.normal((rows, k), 0.5, 2), ref.normal((experts, n, k), 0.05, 3)
    want = (fme.grouped_gemm_fwd_bf16(x, w, off), fme.grouped_gemm_dgrad_bf16(dy, w, off),
            fme.grouped_gemm_wgrad_bf16(dy, x, off))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (fme.grouped_gemm_fwd_bf16(x, w, off, status=status, stream=side),
           fme.grouped_gemm_dgrad_bf16(dy, w, off, status=status, stream=side),
           fme.grouped_gemm_wgrad_bf16(dy, x, off, status=status, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for g, w_ in zip(got, want):
        assert torch.equal(g, w_)
