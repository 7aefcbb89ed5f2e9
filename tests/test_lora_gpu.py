"""Low-rank adapters beside a shared projection, against 64 bits."""
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


def inputs(m, n, k, adapters, rank, dtype, seed, run=1):
    g = torch.Generator().manual_seed(seed)
    x, y = torch.randn(m, k, generator=g).to(dtype), torch.randn(m, n, generator=g).to(dtype)
    a = (torch.randn(adapters, rank, k, generator=g) * k ** -0.5).to(dtype)
    b = torch.randn(adapters, n, rank, generator=g).to(dtype)
    index = torch.randint(-1, adapters, (-(-m // run),), generator=g, dtype=torch.int32).repeat_interleave(run)[:m].contiguous()
    scales = torch.rand(adapters, generator=g) * 2 - 0.5
    return x, y, a, b, index, scales


CASES = [
    # m, n, k, adapters, rank, run, dtype
    (1, 1, 8, 1, 8, 1, "bf16"),
    (1, 2560, 2048, 4, 16, 1, "bf16"),
    (2, 100, 1000, 3, 24, 1, "f16"),
    (15, 257, 136, 20, 8, 1, "bf16"),
    (16, 64, 4096, 16, 32, 1, "f16"),
    (17, 1030, 520, 17, 40, 1, "bf16"),
    (64, 512, 2056, 40, 128, 1, "f16"),
    (70, 333, 128, 1, 64, 70, "bf16"),
    (129, 70, 256, 3, 72, 50, "f16"),
    (1040, 260, 512, 5, 16, 130, "bf16"),
    (1100, 136, 264, 7, 96, 3, "f16"),
]


@pytest.mark.parametrize("scaled", [True, False], ids=["scales", "plain"])
@pytest.mark.parametrize("case", CASES, ids=["m%d_n%d_k%d_l%d_r%d_run%d_%s" % c for c in CASES])
def test_lora_add(dev, case, scaled):
    m, n, k, adapters, rank, run, dts = case
    say("lora", case, scaled)
    lib, dtype = w4(), DT[dts]
    x, y, a, b, index, scales = inputs(m, n, k, adapters, rank, dtype, seed=m + n, run=run)
    if m > 2:
        index[1] = adapters + 5   # no adapter
    s = scales if scaled else None
    want, tol = ref.lora(y, x, a, b, index, s)
    xd, yd, ad, bd, idx = (t.to(dev) for t in (x, y, a, b, index))
    sd = None if s is None else s.to(dev)
    out = lib.lora_add(yd, xd, ad, bd, idx, scales=sd)
    ref.within(out, want, tol, str(case))
    none = (index < 0) | (index >= adapters)
    assert torch.equal(out.cpu()[none], y[none])
    assert torch.equal(yd.cpu(), y), "y changed"
    again = lib.lora_add(yd, xd, ad, bd, idx, scales=sd)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two runs differ"
    got = lib.lora_add(yd, xd, ad, bd, idx, scales=sd, out=yd)
    assert got is yd and torch.equal(yd, out), "in place"


# enough rows and columns for the tiles of 64 rows
LARGE = [
    (1100, 16901, 72, 5, 24, 70, "bf16"),
    (2111, 8200, 264, 7, 128, 300, "f16"),
    (1024, 16384, 40, 9, 64, 1, "bf16"),
    (4100, 4097, 8, 3, 8, 1000, "f16"),
]


@pytest.mark.parametrize("case", LARGE, ids=["m%d_n%d_k%d_l%d_r%d_run%d_%s" % c for c in LARGE])
def test_lora_add_large(dev, case):
    test_lora_add(dev, case, True)


def test_lora_strided_rows(dev):
    say("lora on slices")
    lib = w4()
    for n, off in ((200, 8), (201, 3)):
        x, y, a, b, index, scales = inputs(37, n, 256, 4, 16, torch.bfloat16, 5)
        want, tol = ref.lora(y, x, a, b, index, scales)
        xw = torch.full((37, 272), float("nan"), dtype=torch.bfloat16)
        xw[:, 8:264] = x
        yw = torch.full((37, n + 11), float("nan"), dtype=torch.bfloat16)
        yw[:, off:off + n] = y
        xw, yw = xw.to(dev), yw.to(dev)
        ys = yw[:, off:off + n]
        lib.lora_add(ys, xw[:, 8:264], a.to(dev), b.to(dev), index.to(dev), scales=scales.to(dev), out=ys)
        ref.within(ys, want, tol, f"slices n={n}")
        assert torch.isnan(yw[:, :off]).all() and torch.isnan(yw[:, off + n:]).all()


def test_lora_one_row_does_not_touch_another(dev):
    say("lora with NaN and infinities in other rows and adapters")
    lib = w4()
    x, y, a, b, index, scales = inputs(40, 96, 128, 6, 16, torch.float16, 11)
    index = (torch.arange(40) % 6).to(torch.int32)
    want, tol = ref.lora(y, x, a, b, index, scales)
    bad = torch.zeros(40, dtype=torch.bool)
    x[7], y[9] = float("inf"), float("nan")
    a[4] = float("nan")
    bad[[7, 9]] = True
    bad |= index == 4
    out = lib.lora_add(*(t.to(dev) for t in (y, x, a, b, index)), scales=scales.to(dev)).cpu()
    ref.within(out[~bad], want[~bad], tol[~bad], "rows apart")
    assert not torch.isfinite(out[bad].float()).all(1).any()


def test_lora_range_of_f16(dev):
    say("x A^T beyond f16's range and below its normals")
    lib = w4()
    x, y, a, b, index, _ = inputs(6, 64, 512, 2, 8, torch.float16, 12)
    index = torch.tensor([0, 1, 0, 1, 0, 1], dtype=torch.int32)
    for f, g in ((300.0, 2.0 ** -14), (2.0 ** -12, 1.0)):
        xx, aa, bb = (x * f).to(torch.float16), (a * (300.0 if f > 1 else 1.0)).to(torch.float16), (b * g).to(torch.float16)
        y0 = torch.zeros_like(y)
        want, tol = ref.lora(y0, xx, aa, bb, index, None)
        out = lib.lora_add(*(t.to(dev) for t in (y0, xx, aa, bb, index)))
        ref.within(out, want, tol, f"range {f}")


def test_lora_stream_and_graph(dev):
    say("lora stream and graph")
    lib = w4()
    x, y, a, b, index, scales = (t.to(dev) for t in inputs(33, 520, 1024, 9, 16, torch.bfloat16, 13))
    want = lib.lora_add(y, x, a, b, index, scales=scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = lib.lora_add(y, x, a, b, index, scales=scales)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.zeros(lib.lora_add_workspace_bytes(33, 520, 1024, 9, 16), dtype=torch.uint8, device=dev)
    out = torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lib.lora_add(y, x, a, b, index, scales=scales, out=out, workspace=ws)
    for rep in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
        assert torch.equal(lib.lora_add(y, x, a, b, index, scales=scales), want)
    index.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    assert not ws[:1 << 20].any(), "the workspace's header is not zero"


def test_lora_no_rows(dev):
    say("lora without rows")
    lib = w4()
    x, y, a, b, index, _ = (t.to(dev) for t in inputs(0, 32, 64, 2, 8, torch.bfloat16, 1))
    assert lib.lora_add(y, x, a, b, index).shape == (0, 32)


def test_lora_beside_the_linear(dev):
    say("lora beside the INT4 projection, 3-D input")
    lib = w4()
    g = torch.Generator().manual_seed(3)
    n, k = 272, 512
    packed = lib.pack(*lib.quantize((torch.randn(n, k, generator=g) * 0.02).to(dev)))
    x, _, a, b, _, scales = inputs(10, n, k, 3, 8, torch.bfloat16, 2)
    x = x.view(2, 5, k).to(dev)
    index = torch.tensor([0, 0, 1, -1, 2, 2, 2, 1, 0, -1], dtype=torch.int32, device=dev)
    y = lib.linear(x, packed, n)
    out = lib.lora_add(y, x, a.to(dev), b.to(dev), index, scales=scales.to(dev))
    want, tol = ref.lora(y.cpu().view(10, n), x.cpu().view(10, k), a, b, index.cpu(), scales)
    assert out.shape == (2, 5, n)
    ref.within(out.view(10, n), want, tol, "beside the linear")
