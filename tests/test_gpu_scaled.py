"""The e4m3 quantisers and the block-scaled LM head on the GPU against plain fp64 forms."""
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error(cuda_lib):
    yield
    torch.cuda.synchronize()
    assert cuda_lib.device_error(reset=True) == 0


def _values(seed, rows, cols, dtype):
    """Rows whose blocks span many magnitudes, zeros, exact borders and tiny values among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    x[0, :min(cols, 130)] = 0
    if rows > 2:
        x[1, :16] = 448.0
        x[2, :] = 2.0 ** -140 if dtype == "f32" else 1e-38
    return x.to(ref.TORCH[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (5, 144), (60, 4096), (130, 272)])
def test_quantize(cuda_lib, rows, cols, dtype):
    x = _values(rows + cols, rows, cols, dtype)
    kb = -(-cols // 128)
    x8 = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.full((kb, -(-rows // 4) * 4), 7.0, device="cuda")
    cuda_lib.quantize_rows(x.cuda(), x8, xs)
    want, scale = ref.quantize(x, 1)
    assert torch.equal(x8.cpu().view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(xs.cpu()[:, :rows].double(), scale.t()) and (xs[:, rows:] == 7).all()
    w8 = torch.empty_like(x8)
    ws = torch.empty((-(-rows // 128), kb), device="cuda")
    cuda_lib.quantize_blocks(x.cuda(), w8, ws)
    want, scale = ref.quantize(x, 128)
    assert torch.equal(w8.cpu().view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(ws.cpu().double(), scale)


@pytest.mark.parametrize("rows", [4, 40, 132])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantize_keeps_non_finite_blocks_visible(cuda_lib, bad, rows):
    x = torch.randn(rows, 256)
    x[2, 200] = bad
    x8 = torch.empty((rows, 256), dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.empty((2, rows), device="cuda")
    cuda_lib.quantize_rows(x.cuda(), x8, xs)
    assert torch.isnan(xs.cpu()).nonzero().tolist() == [[1, 2]]
    w8, ws = torch.empty_like(x8), torch.empty((-(-rows // 128), 2), device="cuda")
    cuda_lib.quantize_blocks(x.cuda(), w8, ws)
    assert torch.isnan(ws.cpu()).nonzero().tolist() == [[0, 1]]
    logits = torch.empty((rows, 4), device="cuda")
    y = torch.randn(4, 256)
    y8, ys = torch.empty((4, 256), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((1, 2), device="cuda")
    cuda_lib.quantize_blocks(y.cuda(), y8, ys)
    cuda_lib.lm_head_logits_scaled(x8, xs, y8, ys, logits)
    assert torch.isnan(logits.cpu()).nonzero()[:, 0].unique().tolist() == [2]  # that row alone


def _operands(seed, rows, hidden, vocab):
    g = torch.Generator().manual_seed(seed)
    kb = -(-hidden // 128)
    x8 = torch.randn((rows, hidden), generator=g).mul(60).to(torch.float8_e4m3fn)
    w8 = torch.randn((vocab, hidden), generator=g).mul(60).to(torch.float8_e4m3fn)
    # any fp32 scales, negative and zero ones among them; the padding of x_scales is NaN
    xs = torch.full((kb, -(-rows // 4) * 4), float("nan"))
    xs[:, :rows] = torch.randn((kb, rows), generator=g)
    ws = torch.randn((-(-vocab // 128), kb), generator=g)
    ws[0, 0] = 0
    return x8, xs, w8, ws


SIZES = [  # rows, hidden, vocab
    (1, 16, 1), (1, 128, 128), (2, 144, 129), (1, 4096, 3000), (7, 256, 127), (16, 512, 500), (17, 512, 500),
    (33, 272, 1001), (60, 2048, 1030), (64, 128, 256), (65, 384, 2050), (100, 640, 999), (127, 256, 255),
    (128, 256, 256), (129, 256, 257), (200, 1040, 700), (256, 512, 514), (257, 512, 1026), (300, 128, 3),
    (513, 784, 1300), (1000, 160, 640),
]


@pytest.mark.parametrize("rows,hidden,vocab", SIZES)
def test_scaled_logits(cuda_lib, rows, hidden, vocab):
    ops = _operands(rows * 7 + vocab, rows, hidden, vocab)
    full = torch.full((rows * vocab + 64,), float("nan"), device="cuda")
    logits = full[:rows * vocab].view(rows, vocab)
    d = [t.cuda() for t in ops]
    cuda_lib.lm_head_logits_scaled(*d, logits)
    torch.cuda.synchronize()
    want, bound = ref.logits_scaled(*ops)
    got = logits.double().cpu()
    assert torch.isfinite(got).all() and torch.isnan(full[rows * vocab:]).all()
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound.clamp(min=1e-300)).max()
    again = torch.empty_like(logits)
    cuda_lib.lm_head_logits_scaled(*d, again)
    assert torch.equal(again, logits)


def test_scaled_logits_unaligned_output(cuda_lib):
    """logits need only be 4-byte aligned."""
    for rows, vocab in ((5, 130), (200, 516)):
        ops = _operands(3, rows, 256, vocab)
        full = torch.full((rows * vocab + 8,), float("nan"), device="cuda")
        logits = full[1:1 + rows * vocab].view(rows, vocab)
        cuda_lib.lm_head_logits_scaled(*[t.cuda() for t in ops], logits)
        want, bound = ref.logits_scaled(*ops)
        assert ((logits.double().cpu() - want).abs() <= bound).all()
        assert torch.isnan(full[0]) and torch.isnan(full[1 + rows * vocab:]).all()


@pytest.mark.parametrize("rows", [5, 300])
def test_quantize_then_logits_in_a_graph_and_on_a_stream(cuda_lib, rows):
    """The quantiser's results reach the product that follows it, every time: the pair in a
    replayed graph, its input changed between replays, and on a second stream."""
    H, V = 1024, 2000
    g = torch.Generator().manual_seed(rows)
    w = torch.randn((V, H), generator=g) / 32
    w8 = torch.empty((V, H), dtype=torch.float8_e4m3fn, device="cuda")
    ws = torch.empty((-(-V // 128), H // 128), device="cuda")
    x = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    x8 = torch.empty((rows, H), dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.empty((H // 128, -(-rows // 4) * 4), device="cuda")
    logits = torch.empty((rows, V), device="cuda")
    cuda_lib.quantize_blocks(w.cuda(), w8, ws)

    def pair():
        cuda_lib.quantize_rows(x, x8, xs)
        cuda_lib.lm_head_logits_scaled(x8, xs, w8, ws, logits)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x.copy_(torch.randn((rows, H), generator=g))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pair()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pair()
    for _ in range(4):
        host = torch.randn((rows, H), generator=g).bfloat16()
        x.copy_(host)
        graph.replay()
        torch.cuda.synchronize()
        q, s = ref.quantize(host, 1)
        want, bound = ref.logits_scaled(q, s.t(), w8.cpu(), ws.cpu())
        assert ((logits.double().cpu() - want).abs() <= bound).all()


# ------------------------------------------------------------------ tiles of two vocabulary blocks

# 888 (pair of vocabulary blocks, row tile) pairs and more, which is where these tiles begin:
# odd numbers of blocks, vocabularies that are no multiple of 4 (or of the last block's rows),
# one to four row tiles, more K blocks than the ring has slots and fewer
WIDE = [(129, 640, 113701), (300, 272, 75780), (65, 160, 227301), (385, 1040, 56577), (512, 528, 57000)]


def _wide_reference(ops):
    """As ref.logits_scaled, on the device: the largest take a CPU minutes."""
    return ref.logits_scaled(*[t.cuda() for t in ops])


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("rows,hidden,vocab", WIDE)
def test_scaled_logits_two_blocks(cuda_lib, rows, hidden, vocab, offset):
    blocks = -(-vocab // 128)
    assert (blocks + 1) // 2 * -(-rows // 128) >= 6 * 148
    ops = _operands(rows + vocab, rows, hidden, vocab)
    full = torch.full((rows * vocab + 64,), float("nan"), device="cuda")
    logits = full[offset:offset + rows * vocab].view(rows, vocab)
    d = [t.cuda() for t in ops]
    cuda_lib.lm_head_logits_scaled(*d, logits)
    torch.cuda.synchronize()
    assert torch.isnan(full[:offset]).all() and torch.isnan(full[offset + rows * vocab:]).all()
    want, bound = _wide_reference(ops)
    got = logits.double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound.clamp(min=1e-300)).max()
    again = torch.empty_like(logits)
    cuda_lib.lm_head_logits_scaled(*d, again)
    assert torch.equal(again, logits)


def test_scaled_logits_two_blocks_keep_rows_apart(cuda_lib):
    """A row whose scale is NaN is NaN as a whole, a vocabulary block whose scale is NaN in every
    row; all else is as without them."""
    rows, hidden, vocab = WIDE[0]
    x8, xs, w8, ws = [t.cuda() for t in _operands(4, rows, hidden, vocab)]
    clean, logits = torch.empty((rows, vocab), device="cuda"), torch.empty((rows, vocab), device="cuda")
    cuda_lib.lm_head_logits_scaled(x8, xs, w8, ws, clean)
    xs[2, 100] = xs[4, 128] = ws[888, 0] = ws[301, 3] = float("nan")   # block 888 is the last, alone in its tile
    cuda_lib.lm_head_logits_scaled(x8, xs, w8, ws, logits)
    hit = torch.zeros((rows, vocab), dtype=torch.bool, device="cuda")
    hit[[100, 128]] = True
    hit[:, 888 * 128:] = hit[:, 301 * 128:302 * 128] = True
    assert torch.isfinite(clean).all() and torch.equal(torch.isnan(logits), hit)
    assert torch.equal(logits[~hit], clean[~hit])


# ------------------------------------------------------------------ whole outputs

@pytest.mark.parametrize("rows,hidden,vocab", SIZES + WIDE[:2])
def test_scaled_logits_whole_output(cuda_lib, rows, hidden, vocab):
    """The errors of a whole output, as a root of squares, against its terms'.

    The bound of a single logit counts every rounding at its worst and grows with H; together
    they are random and add as squares.  A block's 128 exact products are summed in four steps
    of 32, each losing at most 2^-23 of a partial sum whose root mean square is the block's at
    most, and its scaling and addition round once each (2^-24, of the sum so far): per block
    sqrt(4) 2^-23 of its own size, and over KB blocks, whose sums grow as the root of their
    number, sqrt(2 KB / 2) 2^-24 of the whole.  For KB <= 32 that is below 2^-21 + 2^-21.4, and
    2^-20 is the limit."""
    ops = _operands(rows * 3 + vocab, rows, hidden, vocab)
    assert -(-hidden // 128) <= 32
    logits = torch.empty((rows, vocab), device="cuda")
    x8, xs, w8, ws = [t.cuda() for t in ops]
    cuda_lib.lm_head_logits_scaled(x8, xs, w8, ws, logits)
    want, _ = _wide_reference(ops)
    x = x8.float().double() * xs[:, :rows].double().t().repeat_interleave(128, 1)[:, :hidden]
    w = w8.float().double() * ws.double().repeat_interleave(128, 0)[:vocab].repeat_interleave(128, 1)[:, :hidden]
    size = ((x * x) @ (w * w).t()).sum().sqrt()   # the root of the terms' squares
    assert (logits.double() - want).norm() <= 2.0 ** -20 * size
