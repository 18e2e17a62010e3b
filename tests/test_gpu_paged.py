"""The paged-cache operators on the GPU against plain fp64 forms (tests/paged_ref.py).

Pools are filled with NaN wherever no sequence keeps a position, and table entries past a
sequence's length hold indices far outside the pool: neither may reach an output."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads as wl
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
JUNK = (-1, 1 << 30, -(1 << 31), 123456789)


@pytest.fixture(autouse=True)
def _no_device_error(cuda_lib):
    yield
    torch.cuda.synchronize()
    assert cuda_lib.device_error(reset=True) == 0


def _normal(g, shape, dtype, gain=1.0):
    return (torch.randn(shape, generator=g) * gain).to(ref.TORCH[dtype])


def _case(seed, B, N, Hq, Hkv, D, page, shared, lens, dtype, copies=False, gain=1.0, max_depth=5, slack=0):
    """CPU tensors of one attention problem.  The first `shared` positions of every sequence
    that is long enough hold the same values: its full pages the same pages (or copies of
    them), the page in which the prefix ends a copy."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    max_len = max(max(lens), shared, 1) + slack
    width = -(-max_len // page)
    need = sum(-(-n // page) for n in lens)
    num = need + 3
    order = torch.randperm(num, generator=g).tolist()
    kp = torch.full((num, Hkv, page, D), float("nan"), dtype=ref.TORCH[dtype])
    vp = torch.full((num, Hkv, page, D), float("inf"), dtype=ref.TORCH[dtype])
    table = torch.tensor([[JUNK[(b + j) % 4] for j in range(width)] for b in range(B)])
    common = [_normal(g, (Hkv, shared, D), dtype, gain) for _ in range(2)]
    first = None
    for b, L in enumerate(lens):
        long = L >= shared
        own = [_normal(g, (Hkv, L, D), dtype, gain) for _ in range(2)]
        if long:
            for o, c in zip(own, common):
                o[:, :shared] = c
        for j in range(-(-L // page)):
            lo, hi = j * page, min(L, (j + 1) * page)
            if long and first is not None and hi <= shared and hi - lo == page and not copies:
                table[b, j] = table[first, j]
                continue
            idx = order.pop()
            table[b, j] = idx
            kp[idx, :, :hi - lo] = own[0][:, lo:hi]
            vp[idx, :, :hi - lo] = own[1][:, lo:hi]
        if long and first is None:
            first = b
    par = np.stack([wl.random_parents(rng, N, max_depth) if N > 1 else np.array([-1]) for _ in range(B)])
    return dict(q=_normal(g, (B, N, Hq, D), dtype, gain), k_pages=kp, v_pages=vp, table=table.to(torch.int32),
                lens=torch.tensor(lens, dtype=torch.int32), k_tree=_normal(g, (B, N, Hkv, D), dtype, gain),
                v_tree=_normal(g, (B, N, Hkv, D), dtype, gain), parents=torch.from_numpy(par.astype(np.int32)),
                shared=shared, max_len=max_len, dtype=dtype)


GUARD = 4096


def _launcher(lib, c, scale=0.0):
    """Device copies, a guarded workspace and output, and the call."""
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    B, N, Hq, D = c["q"].shape
    num, Hkv, page, _ = c["k_pages"].shape
    shape = lib.make_shape(B, N, Hq, Hkv, D, c["max_len"], 64, 128, c["dtype"], scale)
    pages = lib.make_pages(num, page, c["table"].shape[1])
    need = lib.paged_workspace_bytes(shape, pages, c["shared"])
    buf = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    full = torch.full((B * N * Hq * D + 256,), float("nan"), dtype=ref.TORCH[c["dtype"]], device="cuda")
    out = full[:B * N * Hq * D].view(B, N, Hq, D)

    def call(stream=None):
        lib.tree_attention_paged(shape, pages, d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], c["shared"],
                                 d["k_tree"], d["v_tree"], d["parents"], out, buf[:need], stream)

    def guards():
        torch.cuda.synchronize()
        assert (buf[need:] == 0xA5).all() and torch.isnan(full[B * N * Hq * D:]).all()

    return d, out, call, guards


def _check(c, out, scale=None):
    d = c["q"].shape[-1]
    want, bound = ref.attention(c["q"], c["k_pages"], c["v_pages"], c["table"], c["lens"].clamp(0, c["max_len"]),
                                c["k_tree"], c["v_tree"], c["parents"], scale or d ** -0.5, c["dtype"])
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    over = ((got - want).abs() / bound.clamp(min=1e-300)).max().item()
    assert over <= 1.0, f"largest error is {over:.3f} of its bound"


ATTN = [
    # B, N, Hq, Hkv, D, page, shared, lens
    (1, 1, 4, 4, 64, 16, 0, [0]),                               # the token alone
    (1, 1, 8, 2, 128, 16, 0, [1]),
    (2, 1, 32, 8, 128, 16, 0, [127, 128]),
    (3, 1, 6, 3, 128, 32, 0, [129, 0, 257]),
    (1, 1, 32, 8, 128, 16, 0, [4097]),
    (1, 64, 2, 2, 64, 64, 0, [193]),
    (2, 13, 8, 2, 128, 256, 0, [300, 77]),
    (3, 21, 6, 3, 128, 128, 0, [1500, 640, 1]),
    (1, 60, 64, 8, 128, 32, 0, [200]),                          # several row blocks
    (1, 2, 128, 1, 64, 16, 0, [50]),                            # 128 heads share a kv head
    (2, 5, 127, 1, 128, 16, 33, [50, 33]),                      # 127 rows of a tile
    (2, 9, 8, 2, 128, 16, 16, [16, 40]),                        # the prefix ends with a page
    (3, 13, 8, 2, 64, 32, 333, [333, 340, 633]),                # ... inside one
    (4, 60, 8, 2, 128, 16, 130, [131, 300, 130, 1000]),
    (5, 7, 4, 4, 128, 256, 700, [701, 700, 0, 12, 1400]),       # sequences shorter than the prefix
    (3, 4, 4, 4, 128, 16, 50, [0, 3, 49]),                      # none long enough
    (2, 17, 8, 8, 128, 64, 1, [1, 2]),
    (9, 64, 32, 8, 64, 64, 1000, [1000 + 37 * i for i in range(9)]),
    (70, 1, 8, 2, 64, 16, 40, [40 + (i * 29) % 200 for i in range(70)]),
    (4, 64, 8, 2, 128, 256, 0, [63, 64, 65, 192]),              # the tree beside the last keys, or after them
    (4, 7, 4, 4, 64, 128, 40, [40, 104, 105, 128]),
    (33, 3, 4, 2, 128, 16, 0, [(i * 53) % 300 for i in range(33)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"B{c[0]}N{c[1]}H{c[2]}_{c[3]}D{c[4]}p{c[5]}s{c[6]}L{max(c[7])}")
def test_attention(cuda_lib, case, dtype):
    c = _case(len(case[7]) * 1000 + case[1], *case, dtype)
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)


PLAN = [
    # more than 384 sequences, two and three to a thread of the plan: some or none shorter than
    # the shared prefix, empty ones, none that holds it
    (400, 1, 2, 1, 64, 16, 0, [(i * 17) % 41 for i in range(400)]),
    (769, 1, 4, 2, 64, 16, 20, [(i * 17) % 61 for i in range(769)]),
    (800, 2, 4, 1, 128, 16, 33, [33 + (i * 31) % 300 for i in range(800)]),
    (385, 1, 2, 1, 128, 32, 50, [(i * 13) % 50 for i in range(385)]),
    # three row tiles of a sequence and 43 of the batch: pairs and single tiles in turn on a CTA
    (17, 40, 64, 8, 64, 64, 200, [200 + 300 + (i * 397) % 1000 for i in range(17)]),
    (6, 41, 16, 2, 128, 16, 300, [300 + (i * 397) % 1000 for i in range(6)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", PLAN, ids=lambda c: f"B{c[0]}N{c[1]}H{c[2]}_{c[3]}D{c[4]}p{c[5]}s{c[6]}L{max(c[7])}")
def test_attention_large_batches_and_odd_row_tiles(cuda_lib, case, dtype):
    c = _case(len(case[7]) * 1000 + case[1], *case, dtype)
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)
    first = out.clone()
    for _ in range(3):
        out.fill_(7.0)
        call()
        assert torch.equal(out, first)


@pytest.mark.parametrize("case", ATTN + PLAN, ids=lambda c: f"B{c[0]}N{c[1]}H{c[2]}_{c[3]}D{c[4]}p{c[5]}s{c[6]}L{max(c[7])}")
def test_attention_f32_whole_output(cuda_lib, case):
    """The errors of a whole fp32 output, as a root of squares, against the output's.

    A score's D-long chain of multiply-adds has partial sums that grow as the root of their
    number: together they lose sqrt(D / 2) 2^-24 of a score of about 1.  The scaled score, its
    difference from the maximum (magnitudes up to about 4) and the exponential round by at most
    6 2^-24 more, the n-long sum over the keys by sqrt(n / 2) 2^-24; the rescalings of the
    running sums and the merge belong to that count.  Twice their sum is the limit."""
    c = _case(len(case[7]) * 77 + case[1], *case, "f32")
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    B, N, Hq, D = c["q"].shape
    want, _ = ref.attention(c["q"], c["k_pages"], c["v_pages"], c["table"], c["lens"], c["k_tree"], c["v_tree"],
                            c["parents"], D ** -0.5, "f32")
    n = max(case[7]) + N
    limit = 2 * 2.0 ** -24 * ((D / 2) ** 0.5 + 6 + (n / 2) ** 0.5)
    assert (out.double().cpu() - want).norm() <= limit * want.norm()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_copied_prefix_large_values_and_scale(cuda_lib, dtype):
    """Copies of the shared pages; scores spread so widely that rows rest on a few keys and
    running maxima jump; a softmax scale of the caller's."""
    c = _case(5, 3, 12, 8, 4, 128, 32, 300, [300, 411, 1200], dtype, copies=True, gain=3.0, slack=500)
    _, out, call, guards = _launcher(cuda_lib, c, scale=0.25)
    call()
    guards()
    _check(c, out, 0.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rising_scores(cuda_lib, dtype):
    """Keys whose scores grow along the prefix: every tile lifts the running maximum."""
    c = _case(6, 2, 5, 4, 4, 64, 16, 256, [900, 700], dtype)
    for b in range(2):
        for j in range(-(-int(c["lens"][b]) // 16)):
            c["k_pages"][c["table"][b, j]] = (0.004 * j) * torch.ones(64).to(c["k_pages"].dtype)
    c["q"].fill_(2.0)
    c["k_pages"] = torch.where(torch.isfinite(c["k_pages"]), c["k_pages"], torch.zeros_like(c["k_pages"]))
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [0, 200])
def test_attention_bad_page_counts_as_zero(cuda_lib, dtype, shared):
    c = _case(7, 2, 5, 8, 2, 128, 32, shared, [300, 260], dtype, copies=True)
    c["table"][1, 7] = c["k_pages"].shape[0]       # own part: positions 224 ..
    if shared:
        c["table"][0, 2] = c["table"][1, 2] = -3   # shared part: positions 64 .. of either
    else:
        c["table"][0, 2] = -3
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)
    assert cuda_lib.device_error(reset=True) == 0x206


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_length_outside_is_clamped_and_recorded(cuda_lib, dtype):
    c = _case(8, 3, 5, 4, 2, 64, 16, 32, [160, 0, 77], dtype)
    c["lens"][0], c["lens"][1] = 100000, -4        # clamped to max_len = 160 and to 0
    assert c["max_len"] == 160
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)
    assert cuda_lib.device_error(reset=True) == 0x205


def test_attention_invalid_parent_ends_the_path(cuda_lib):
    c = _case(9, 1, 6, 4, 2, 128, 16, 0, [70], "bf16")
    c["parents"][0, 3] = 5      # forward link
    c["parents"][0, 4] = -7
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_repeats_bit_for_bit_on_streams_and_in_graphs(cuda_lib, dtype):
    """The same bits on the default stream, on another one, and from a replayed graph whose
    inputs changed after the capture; a workspace full of another call's values does not
    matter."""
    c = _case(10, 4, 20, 8, 2, 128, 16, 100, [100, 900, 350, 20], dtype)
    d, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([900, 100, 0, 350], [100, 900, 350, 20]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        order = [c["lens"].tolist().index(n) if n in c["lens"].tolist() else 3 for n in lens]
        d["table"].copy_(c["table"][order])
        graph.replay()
        guards()
        c2 = dict(c, lens=torch.tensor(lens, dtype=torch.int32), table=c["table"][order])
        _check(c2, out)
    assert torch.equal(out, first)


def test_attention_ragged_batch_repeats(cuda_lib):
    """Short sequences of every length, so that runs of single tiles follow one another on a
    CTA: the same bits every time, with other memory traffic in between."""
    c = _case(33003, *ATTN[-1], "bf16")
    _, out, call, guards = _launcher(cuda_lib, c)
    call()
    guards()
    _check(c, out)
    first = out.clone()
    junk = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for i in range(60):
        out.fill_(7.0)
        if i % 3 == 0:
            junk.fill_(i)
        call()
        assert torch.equal(out, first), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [0, 40])
def test_attention_nan_reaches_those_that_see_it(cuda_lib, dtype, shared):
    """A NaN in one key: every output that sees the key is NaN, wherever it falls in a tile
    and though it may be alone in its part; all others are as without it."""
    clean = _case(14, 3, 9, 4, 2, 64, 16, shared, [300, 0, 41], dtype)
    _, out, call, guards = _launcher(cuda_lib, clean)
    call()
    guards()
    _check(clean, out)
    keys = [("prefix", 0, 45), ("prefix", 0, 128), ("prefix", 0, 299), ("prefix", 2, 40)]
    keys += [("prefix", 0, j) for j in range(130, 150)] + [("tree", b, i) for b in range(3) for i in range(9)]
    for kind, b, i in keys:
        c = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in clean.items()}
        hit = torch.zeros(out.shape, dtype=torch.bool)
        if kind == "tree":
            c["k_tree"][b, i, 1] = float("nan")
            hit[b, :, 2:] = ref.visible(c["parents"][b].tolist())[:, i, None, None]
        else:
            c["k_pages"][c["table"][b, i // 16], 1, i % 16] = float("nan")
            hit[b, :, 2:] = True
        _, got, call, guards = _launcher(cuda_lib, c)
        call()
        guards()
        assert torch.equal(torch.isnan(got).cpu(), hit), (kind, b, i)
        assert torch.equal(got[~hit.cuda()], out[~hit.cuda()]), (kind, b, i)


FIRST_CALL = """
import sys
import torch
from tests import test_gpu_paged as t
from tree_verify_b200 import binding
dtype = sys.argv[1]
c = t._case(15, 2, 9, 4, 2, 128, 16, 30, [300, 31], dtype)
_, out, call, guards = t._launcher(binding, c)
x = torch.randn((33, 256), device="cuda")
w = torch.randn((300, 256), device="cuda")
e4m3 = torch.float8_e4m3fn
x8, w8 = torch.empty(x.shape, dtype=e4m3, device="cuda"), torch.empty(w.shape, dtype=e4m3, device="cuda")
xs, ws = torch.empty((2, 36), device="cuda"), torch.empty((3, 2), device="cuda")
logits = torch.empty((33, 300), device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
    binding.quantize_blocks(w, w8, ws)
    binding.quantize_rows(x, x8, xs)
    binding.lm_head_logits_scaled(x8, xs, w8, ws, logits)
for _ in range(2):
    graph.replay()
guards()
t._check(c, out)
first = logits.clone()
binding.lm_head_logits_scaled(x8, xs, w8, ws, logits)
torch.cuda.synchronize()
assert torch.equal(first, logits) and torch.isfinite(logits).all()
assert binding.device_error(reset=True) == 0
"""


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_first_calls_of_a_process_may_be_captured(dtype):
    done = subprocess.run([sys.executable, "-c", FIRST_CALL, dtype], cwd=ROOT, capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_attention_two_calls_at_once(cuda_lib):
    """Two calls on two streams, each with its own workspace."""
    a = _case(11, 3, 30, 8, 2, 128, 16, 64, [2000, 64, 700], "bf16")
    b = _case(12, 2, 30, 8, 2, 128, 64, 0, [1900, 1000], "bf16")
    _, out_a, call_a, guards_a = _launcher(cuda_lib, a)
    _, out_b, call_b, guards_b = _launcher(cuda_lib, b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        call_a(sa)
        call_b(sb)
    guards_a()
    guards_b()
    _check(a, out_a)
    _check(b, out_b)


def test_attention_pool_offsets_past_32_bits(cuda_lib):
    """Pages at the end of a pool of more than 2^31 elements (and 2^32 bytes)."""
    c = _case(13, 1, 3, 8, 8, 128, 256, 0, [600], "bf16")
    num = (1 << 31) // (8 * 256 * 128) + 4
    big = [torch.empty((num, 8, 256, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = c["table"].clone()
    for j in range(3):
        src = int(c["table"][0, j])
        table[0, j] = num - 1 - j
        big[0][num - 1 - j].copy_(c["k_pages"][src])
        big[1][num - 1 - j].copy_(c["v_pages"][src])
    shape = cuda_lib.make_shape(1, 3, 8, 8, 128, 600, 64, 128, "bf16")
    pages = cuda_lib.make_pages(num, 256, c["table"].shape[1])
    ws = torch.empty(max(256, cuda_lib.paged_workspace_bytes(shape, pages, 0)), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, 3, 8, 128), dtype=torch.bfloat16, device="cuda")
    cuda_lib.tree_attention_paged(shape, pages, c["q"].cuda(), *big, table.cuda(), c["lens"].cuda(), 0,
                                  c["k_tree"].cuda(), c["v_tree"].cuda(), c["parents"].cuda(), out, ws)
    torch.cuda.synchronize()
    _check(c, out)


# ------------------------------------------------------------------ append

def _append_case(seed, B, Hq, Hkv, D, page, rd, interleaved, dtype, rows, packed):
    g = torch.Generator().manual_seed(seed)
    table_len = 400
    width = -(-table_len // page)
    num = B * width + 2
    table = torch.randperm(num, generator=g)[:B * width].view(B, width).to(torch.int32)
    # distinct slots, some padding rows (position -1), some rows that are only rotated
    slots = torch.randperm(B * table_len, generator=g)[:rows]
    seq, pos = (slots // table_len).to(torch.int32), (slots % table_len).to(torch.int32)
    for r in range(rows):
        if r % 7 == 3:
            pos[r] = -1 - r
        elif r % 7 == 5:
            seq[r] = -1
    wide = (Hq + 2 * Hkv) * D
    dt = ref.TORCH[dtype]
    if packed:
        qkv = torch.randn((rows, wide + 16), generator=g).to(dt)  # a gap behind every row
        q, k, v = (qkv[:, a:a + h * D].unflatten(1, (h, D)) for a, h in
                   ((0, Hq), (Hq * D, Hkv), ((Hq + Hkv) * D, Hkv)))
    else:
        q, k, v = (torch.randn((rows, h, D), generator=g).to(dt) for h in (Hq, Hkv, Hkv))
    angle = torch.rand((table_len, rd // 2), generator=g, dtype=torch.float64) * 6.28
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    pools = [torch.randn((num, Hkv, page, D), generator=g).to(dt) for _ in range(2)]
    return dict(q=q, k=k, v=v, pos=pos, seq=seq, cs=cs, table=table, kp=pools[0], vp=pools[1], B=B, rd=rd,
                il=interleaved, dtype=dtype, page=page)


def _strided(t):
    """A device copy that keeps the strides (row gaps filled with NaN)."""
    buf = torch.full((t.shape[0] * t.stride(0) + 8,), float("nan"), dtype=t.dtype, device="cuda")
    out = buf.as_strided(t.shape, t.stride())
    out.copy_(t)
    return out


def _check_rotated(got, x, cos, sin, c, live):
    want, bound = ref.rotate(x, cos, sin, c["rd"], c["il"])
    bound = bound + ref.HALF_STEP[c["dtype"]] * (want.abs() + bound)
    err = (got.double().cpu() - want).abs()
    assert (err[live] <= bound[live]).all()
    keep = got.cpu()[..., c["rd"]:][live]
    assert torch.equal(keep, x[..., c["rd"]:][live])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("geom", [
    # B, Hq, Hkv, D, page, rotary, interleaved, rows, packed
    (1, 4, 4, 64, 16, 64, False, 1, False),
    (3, 8, 2, 128, 16, 128, False, 50, True),
    (2, 6, 3, 128, 64, 64, False, 33, True),
    (2, 8, 2, 64, 256, 32, True, 40, True),
    (4, 5, 1, 128, 32, 128, True, 200, False),
    (2, 2, 2, 128, 128, 16, False, 9, False),
    (2, 2, 2, 64, 16, 48, True, 9, True),
    (2, 64, 8, 128, 16, 0, False, 12, True),
], ids=str)
def test_append(cuda_lib, geom, dtype):
    B, Hq, Hkv, D, page, rd, il, rows, packed = geom
    c = _append_case(rows * 100 + D, B, Hq, Hkv, D, page, rd, il, dtype, rows, packed)
    shape = cuda_lib.make_shape(B, 1, Hq, Hkv, D, 400, 64, 128, dtype)
    pages = cuda_lib.make_pages(c["kp"].shape[0], page, c["table"].shape[1])
    q, k, v = (_strided(c[n]) for n in "qkv")
    kp, vp = c["kp"].cuda(), c["vp"].cuda()
    q_out = torch.full((rows, Hq, D), 7.0, dtype=c["q"].dtype, device="cuda")
    k_out = torch.full((rows, Hkv, D), 7.0, dtype=c["q"].dtype, device="cuda")
    cuda_lib.rope_append(shape, pages, q, k, v, c["pos"].cuda(), c["seq"].cuda(), c["cs"].cuda() if rd else None,
                         kp, vp, c["table"].cuda(), q_out, k_out, interleaved=il)
    torch.cuda.synchronize()
    live = c["pos"] >= 0
    at = c["pos"].clamp(min=0).long()
    cos, sin = c["cs"][at, :rd // 2], c["cs"][at, rd // 2:]
    _check_rotated(q_out, c["q"], cos, sin, c, live)
    _check_rotated(k_out, c["k"], cos, sin, c, live)
    assert (q_out.cpu()[~live] == 7).all() and (k_out.cpu()[~live] == 7).all()
    # the pools: the rotated keys (the bits of k_out) and the values in their slots, all else kept
    wk, wv = c["kp"].clone(), c["vp"].clone()
    for r in range(rows):
        if live[r] and c["seq"][r] >= 0:
            p = int(c["pos"][r])
            idx = int(c["table"][c["seq"][r], p // page])
            wk[idx, :, p % page] = k_out.cpu()[r]
            wv[idx, :, p % page] = c["v"][r]
    assert torch.equal(kp.cpu(), wk) and torch.equal(vp.cpu(), wv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_in_place_and_parts(cuda_lib, dtype):
    """Outputs over their own inputs, queries alone, keys alone without a cache."""
    c = _append_case(3, 2, 4, 2, 64, 16, 64, False, dtype, 20, False)
    shape = cuda_lib.make_shape(2, 1, 4, 2, 64, 400, 64, 128, dtype)
    pages = cuda_lib.make_pages(c["kp"].shape[0], 16, c["table"].shape[1])
    pos, seq, cs, table = (c[n].cuda() for n in ("pos", "seq", "cs", "table"))
    q, k, v, kp, vp = (c[n].cuda() for n in ("q", "k", "v", "kp", "vp"))
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    cuda_lib.rope_append(shape, pages, q, k, v, pos, seq, cs, kp, vp, table, q_out, k_out)
    live = (c["pos"] >= 0).cuda()
    only_q, only_k = torch.zeros_like(q), torch.zeros_like(k)
    cuda_lib.rope_append(shape, None, q, None, None, pos, None, cs, None, None, None, only_q)
    cuda_lib.rope_append(shape, None, None, k, None, pos, None, cs, None, None, None, None, only_k)
    kp2, vp2 = c["kp"].cuda(), c["vp"].cuda()
    cuda_lib.rope_append(shape, pages, None, k, v, pos, seq, cs, kp2, vp2, table, None)
    assert torch.equal(only_q, q_out) and torch.equal(only_k, k_out)
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)
    cuda_lib.rope_append(shape, None, q, k, None, pos, None, cs, None, None, None, q, k)
    assert torch.equal(q[live], q_out[live]) and torch.equal(k[live], k_out[live])
    assert torch.equal(q[~live].cpu(), c["q"][~live.cpu()])


def test_append_bad_rows_are_skipped_whole(cuda_lib):
    c = _append_case(4, 2, 4, 2, 128, 16, 128, False, "bf16", 6, False)
    c["pos"] = torch.tensor([5, 399, 400, 10, 11, 12], dtype=torch.int32)
    c["seq"] = torch.tensor([0, 1, 0, 2, -2, 1], dtype=torch.int32)
    shape = cuda_lib.make_shape(2, 1, 4, 2, 128, 400, 64, 128, "bf16")
    pages = cuda_lib.make_pages(c["kp"].shape[0], 16, c["table"].shape[1])
    kp, vp = c["kp"].cuda(), c["vp"].cuda()
    q_out = torch.full((6, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")

    def call():
        cuda_lib.rope_append(shape, pages, c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), c["pos"].cuda(),
                             c["seq"].cuda(), c["cs"].cuda(), kp, vp, c["table"].cuda(), q_out)
        torch.cuda.synchronize()

    call()
    assert cuda_lib.device_error(reset=True) == 0x401
    assert (q_out[[2, 3, 4]] == 7).all() and not (q_out[[0, 1, 5]] == 7).all()
    changed = (kp.cpu() != c["kp"]).any(-1).any(1).nonzero().tolist()
    want = sorted([[int(c["table"][0, 0]), 5], [int(c["table"][1, 24]), 15], [int(c["table"][1, 0]), 12]])
    assert sorted(changed) == want
    # a position past the cache but inside the angle table, and a page outside the pool
    c["pos"] = torch.tensor([-1, -1, -1, -1, -1, 30], dtype=torch.int32)
    c["table"][1, 1] = -1
    q_out.fill_(7)
    call()
    assert cuda_lib.device_error(reset=True) == 0x206 and (q_out == 7).all()
    pages = cuda_lib.make_pages(c["kp"].shape[0], 16, 1)   # a table of one page a sequence
    c["table"] = c["table"][:, :1].contiguous()
    call()
    assert cuda_lib.device_error(reset=True) == 0x401 and (q_out == 7).all()


def test_append_rows_behind_the_last(cuda_lib):
    """num_rows 0, and a call whose rows are all padding: nothing changes."""
    c = _append_case(5, 1, 4, 2, 64, 16, 64, False, "bf16", 4, False)
    shape = cuda_lib.make_shape(1, 1, 4, 2, 64, 400, 64, 128, "bf16")
    pages = cuda_lib.make_pages(c["kp"].shape[0], 16, c["table"].shape[1])
    kp, vp = c["kp"].cuda(), c["vp"].cuda()
    q_out = torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    junk = torch.full((4,), 1 << 30, dtype=torch.int32, device="cuda")
    for n in (4, 0):
        cuda_lib.rope_append(shape, pages, c["q"].cuda()[:n], c["k"].cuda()[:n], c["v"].cuda()[:n], pos[:n], junk[:n],
                             c["cs"].cuda(), kp, vp, c["table"].cuda(), q_out[:n])
    torch.cuda.synchronize()
    assert (q_out == 7).all() and torch.equal(kp.cpu(), c["kp"]) and torch.equal(vp.cpu(), c["vp"])


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("geom", [(1, 1, 1, 64, 16, 8), (5, 13, 2, 128, 16, 256), (40, 64, 4, 64, 64, 136),
                                  (3, 60, 8, 128, 256, 1024)], ids=str)
def test_commit(cuda_lib, geom, dtype):
    """Random accepted paths with every refused kind among them: an invalid tree (-1), a path
    that is no chain, a node outside the tree, a length outside the cache, no room, a page
    outside the pool."""
    B, N, Hkv, D, page, H = geom
    rng = np.random.default_rng(B * 100 + N)
    g = torch.Generator().manual_seed(B * 100 + N)
    width = -(-(300 + N) // page)
    cap = width * page
    num = B * width + 1
    table = torch.randperm(num, generator=g)[:B * width].view(B, width).to(torch.int32)
    par = np.stack([wl.random_parents(rng, N, 9) if N > 1 else np.array([-1]) for _ in range(B)]).astype(np.int32)
    acc = np.full((B, N), -1, np.int32)
    alen = np.zeros(B, np.int32)
    lens = rng.integers(0, 300, B).astype(np.int32)
    want_len = np.zeros(B, np.int32)
    recorded = False
    for b in range(B):
        path, a = [], int(rng.integers(0, N))
        while a > 0:
            path.append(a)
            a = int(par[b, a])
        path = path[::-1]
        acc[b, :len(path)], alen[b] = path, len(path)
        want_len[b] = lens[b] + len(path) + 1
        kind = b % 9
        if kind == 3:
            alen[b], want_len[b] = -1, lens[b]
        elif kind == 4 and path:
            acc[b, len(path) - 1] = 0
            want_len[b] = -1
        elif kind == 5:
            lens[b] = cap - len(path)          # room for one row too few
            want_len[b] = -1
        elif kind == 6:
            alen[b], want_len[b] = N, -1
        elif kind == 7:
            lens[b], want_len[b] = -5, -1
        elif kind == 8:
            table[b, int(lens[b]) // page], want_len[b] = num, -1
            recorded = True
        elif kind == 2:
            lens[b] = cap - len(path) - 1      # ends with the cache
            want_len[b] = cap
    dt = ref.TORCH[dtype]
    t = dict(kp=torch.randn((num, Hkv, page, D), generator=g).to(dt), vp=torch.randn((num, Hkv, page, D), generator=g).to(dt),
             kt=torch.randn((B, N, Hkv, D), generator=g).to(dt), vt=torch.randn((B, N, Hkv, D), generator=g).to(dt),
             hidden=torch.randn((B * N, H), generator=g).to(dt))
    d = {k: v.cuda() for k, v in t.items()}
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    new = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    feat = torch.full((B, N, H), 7.0, dtype=dt, device="cuda")
    shape = cuda_lib.make_shape(B, N, Hkv * 2, Hkv, D, 16, H, 128, dtype)
    cuda_lib.commit_accepted_paged(shape, cuda_lib.make_pages(num, page, width), d["kp"], d["vp"], table.cuda(),
                                   i32(lens), d["kt"], d["vt"], d["hidden"], i32(par), i32(acc), i32(alen), new, feat)
    torch.cuda.synchronize()
    assert np.array_equal(new.cpu().numpy(), want_len)
    wf = torch.full((B, N, H), 7.0, dtype=dt)
    for b in range(B):
        if want_len[b] < 0 or alen[b] < 0:
            continue
        for i, node in enumerate([0] + acc[b, :alen[b]].tolist()):
            p = int(lens[b]) + i
            idx = int(table[b, p // page])
            t["kp"][idx, :, p % page], t["vp"][idx, :, p % page] = t["kt"][b, node], t["vt"][b, node]
            wf[b, i] = t["hidden"][b * N + node]
    assert torch.equal(d["kp"].cpu(), t["kp"]) and torch.equal(d["vp"].cpu(), t["vp"])
    assert torch.equal(feat.cpu(), wf)
    assert cuda_lib.device_error(reset=True) == (0x206 if recorded else 0)


# ------------------------------------------------------------------ tensors that do not fit

def test_tensors_that_do_not_fit_are_refused(cuda_lib):
    """Sizes, types and layouts that the shape contradicts never reach the library."""
    c = _case(14, 2, 3, 4, 2, 64, 16, 0, [40, 20], "bf16")
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    shape = cuda_lib.make_shape(2, 3, 4, 2, 64, 40, 64, 128, "bf16")
    pages = cuda_lib.make_pages(d["k_pages"].shape[0], 16, d["table"].shape[1])
    ws = torch.empty(cuda_lib.paged_workspace_bytes(shape, pages, 0), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d["q"])
    args = dict(q=d["q"], k_pages=d["k_pages"], v_pages=d["v_pages"], page_table=d["table"], prefix_lens=d["lens"],
                shared_len=0, k_tree=d["k_tree"], v_tree=d["v_tree"], parents=d["parents"], out=out, workspace=ws)
    call = lambda **kw: cuda_lib.tree_attention_paged(shape, pages, **{**args, **kw})
    call()
    for name in ("q", "k_pages", "v_pages", "k_tree", "v_tree", "out"):
        for bad in (args[name].float(), args[name][:1].contiguous(), args[name].cpu(),
                    args[name].transpose(1, 2)):
            with pytest.raises(ValueError):
                call(**{name: bad})
    for name in ("page_table", "prefix_lens", "parents"):
        for bad in (args[name].long(), args[name][:1].contiguous(), args[name].cpu()):
            with pytest.raises(ValueError):
                call(**{name: bad})
    with pytest.raises(cuda_lib.EagleError):
        call(workspace=ws[:256])
    with pytest.raises(cuda_lib.EagleError):
        call(workspace=None)
    with pytest.raises(ValueError):
        call(workspace=ws.view(torch.float32))
    with pytest.raises(cuda_lib.EagleError):
        call(shared_len=41)
    # rows of an append
    R = 5
    q, k = torch.zeros((R, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((R, 2, 64), dtype=torch.bfloat16,
                                                                                     device="cuda")
    pos = torch.zeros((R,), dtype=torch.int32, device="cuda")
    cs = torch.zeros((40, 64), device="cuda")
    rope = lambda **kw: cuda_lib.rope_append(shape, pages, **{**dict(
        q=q, k=k, v=k.clone(), positions=pos, seq_ids=torch.full_like(pos, -1), cos_sin=cs, k_pages=d["k_pages"],
        v_pages=d["v_pages"], page_table=d["table"], q_out=torch.empty_like(q)), **kw})
    rope()
    for kw in (dict(q=q[:4]), dict(q=q.float()), dict(k=k[:, :1]), dict(v=k.transpose(1, 2)), dict(positions=pos[:4]),
               dict(seq_ids=pos[:4]), dict(positions=pos.long()), dict(cos_sin=cs.double()), dict(cos_sin=cs[0]),
               dict(q_out=torch.empty_like(q)[:4]), dict(k_out=torch.empty_like(q)), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            rope(**kw)
    with pytest.raises(cuda_lib.EagleError):
        rope(cos_sin=torch.zeros((40, 72), device="cuda"))       # wider than a head
    # logits
    x8 = torch.zeros((3, 256), dtype=torch.float8_e4m3fn, device="cuda")
    w8, ws8 = torch.zeros((128, 256), dtype=torch.float8_e4m3fn, device="cuda"), torch.ones((1, 2), device="cuda")
    xs, logits = torch.ones((2, 4), device="cuda"), torch.empty((3, 128), device="cuda")
    cuda_lib.lm_head_logits_scaled(x8, xs, w8, ws8, logits)
    cuda_lib.lm_head_logits_scaled(x8.view(torch.uint8), xs, w8.view(torch.uint8), ws8, logits)  # their bytes
    for bad in ((x8.float(), xs, w8, ws8, logits), (x8, xs[:1], w8, ws8, logits), (x8, xs, w8.half(), ws8, logits),
                (x8, xs, w8, ws8.double(), logits), (x8, xs, w8, ws8, logits.half()), (x8, xs, w8[:64], ws8, logits)):
        with pytest.raises(ValueError):
            cuda_lib.lm_head_logits_scaled(*bad)


def test_tensors_in_another_order_are_refused(cuda_lib):
    """Dense tensors of the right size whose dimensions are swapped; merged or split dimensions
    are the same memory and are taken."""
    B, N, Hq, Hkv, D, H = 2, 3, 4, 2, 64, 64
    c = _case(16, B, N, Hq, Hkv, D, 16, 0, [40, 20], "bf16")
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    shape = cuda_lib.make_shape(B, N, Hq, Hkv, D, 40, H, 128, "bf16")
    num = d["k_pages"].shape[0]
    pages = cuda_lib.make_pages(num, 16, d["table"].shape[1])
    ws = torch.empty(cuda_lib.paged_workspace_bytes(shape, pages, 0), dtype=torch.uint8, device="cuda")
    args = dict(q=d["q"], k_pages=d["k_pages"], v_pages=d["v_pages"], page_table=d["table"], prefix_lens=d["lens"],
                shared_len=0, k_tree=d["k_tree"], v_tree=d["v_tree"], parents=d["parents"],
                out=torch.empty_like(d["q"]), workspace=ws)
    call = lambda **kw: cuda_lib.tree_attention_paged(shape, pages, **{**args, **kw})
    swap = lambda t: t.transpose(-3, -2).contiguous() if t.dim() > 2 else t.t().contiguous()
    call()
    for name in ("q", "k_tree", "v_tree", "k_pages", "v_pages", "out", "page_table", "parents"):
        other = swap(args[name])
        for bad in (other, other.flatten(0, 1)) if other.dim() == 4 else (other,):
            with pytest.raises(ValueError):
                call(**{name: bad})
    for q, kt, kp in ((d["q"].view(B * N, Hq, D), d["k_tree"].view(B, N, -1), d["k_pages"].view(num * Hkv, 16, D)),
                      (d["q"].view(B, N, Hkv, Hq // Hkv, D), d["k_tree"].view(-1), d["k_pages"].view(num, Hkv, -1)),
                      (d["q"].view(B * N, Hkv, Hq // Hkv, D), d["k_tree"][None], d["k_pages"].view(1, num, Hkv, 16, 1, D))):
        out = torch.empty_like(q)
        call(q=q, k_tree=kt, k_pages=kp, out=out)
        assert torch.equal(out.view(-1), args["out"].view(-1))
    # append: the rotated keys as [heads, R, D]
    k, pos = torch.zeros((5, Hkv, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((5,), dtype=torch.int32, device="cuda")
    cs = torch.zeros((40, D), device="cuda")
    rope = lambda k_out: cuda_lib.rope_append(shape, None, None, k, None, pos, None, cs, None, None, None, None, k_out)
    rope(torch.empty_like(k).view(5, -1))
    with pytest.raises(ValueError):
        rope(torch.empty((Hkv, 5, D), dtype=torch.bfloat16, device="cuda"))
    # commit: hidden rows and features as [N, B, H], paths as [N, B]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    rows = torch.zeros((B * N, H), dtype=torch.bfloat16, device="cuda")
    commit = lambda hidden, acc, feat: cuda_lib.commit_accepted_paged(
        shape, pages, d["k_pages"], d["v_pages"], d["table"], i32(B), d["k_tree"], d["v_tree"], hidden, d["parents"], acc,
        torch.full((B,), -1, dtype=torch.int32, device="cuda"), i32(B), feat)
    commit(rows, i32(B, N), torch.zeros_like(rows).view(B, N, H))
    commit(rows.view(B, N, H), i32(B * N), torch.zeros_like(rows))
    for bad in ((rows.view(N, B, H), i32(B, N), torch.zeros_like(rows)), (rows, i32(N, B), torch.zeros_like(rows)),
                (rows, i32(B, N), torch.zeros_like(rows).view(N, B, H))):
        with pytest.raises(ValueError):
            commit(*bad)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_run_of_steps(cuda_lib, dtype):
    """Two sequences behind a common prompt: the prompt appended once and its pages shared,
    then three verification steps (the tree's queries and keys rotated at their positions,
    attention over the shared prefix, logits, the greedy walk, the commit) and a decoding
    step, every attention against the fp64 form on an unpaged history."""
    B, N, Hq, Hkv, D, page, H, V = 2, 7, 4, 2, 64, 16, 256, 640
    g = torch.Generator().manual_seed(21)
    dt = ref.TORCH[dtype]
    rand = lambda *s: torch.randn(s, generator=g).to(dt)
    table_len, width, prompt = 128, 8, 37
    freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    angle = torch.arange(table_len, dtype=torch.float64)[:, None] * freq
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    cs_d = cs.cuda()
    num = 2 * width
    kp = torch.full((num, Hkv, page, D), float("nan"), dtype=dt, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    table = torch.arange(num, dtype=torch.int32).view(B, width)
    table[1, :prompt // page] = table[0, :prompt // page]
    table_d = table.cuda()
    shape = cuda_lib.make_shape(B, N, Hq, Hkv, D, width * page, H, V, dtype)
    pages = cuda_lib.make_pages(num, page, width)
    one = cuda_lib.make_shape(B, 1, Hq, Hkv, D, width * page, H, V, dtype)
    ws = torch.empty(max(256, cuda_lib.paged_workspace_bytes(shape, pages, prompt),
                         cuda_lib.paged_workspace_bytes(one, pages, prompt)), dtype=torch.uint8, device="cuda")
    # the prompt: its rows once for sequence 0; for sequence 1 the rows of the page the two part in
    pk, pv = rand(prompt, Hkv, D), rand(prompt, Hkv, D)
    pos = list(range(prompt)) + list(range(prompt // page * page, prompt))
    seq = [0] * prompt + [1] * (len(pos) - prompt)
    k_out = torch.empty((len(pos), Hkv, D), dtype=dt, device="cuda")
    cuda_lib.rope_append(shape, pages, None, torch.cat([pk, pk[prompt // page * page:]]).cuda(),
                         torch.cat([pv, pv[prompt // page * page:]]).cuda(),
                         torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(seq, dtype=torch.int32).cuda(), cs_d,
                         kp, vp, table_d, None, k_out)
    hist_k = [k_out[:prompt].cpu() for _ in range(B)]
    hist_v = [pv.clone() for _ in range(B)]
    lens = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros_like(lens)
    w = torch.randn((V, H), generator=g) / 16
    w8 = torch.empty((V, H), dtype=torch.float8_e4m3fn, device="cuda")
    wscale = torch.empty((V // 128, H // 128), dtype=torch.float32, device="cuda")
    cuda_lib.quantize_blocks(w.cuda(), w8, wscale)
    M = B * N
    x8 = torch.empty((M, H), dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.empty((H // 128, -(-M // 4) * 4), dtype=torch.float32, device="cuda")
    logits = torch.empty((M, V), dtype=torch.float32, device="cuda")
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2, 3]] * B, dtype=torch.int32)
    depth = torch.tensor([0, 1, 1, 2, 2, 2, 3])
    acc = torch.empty((B, N), dtype=torch.int32, device="cuda")
    alen, nxt = torch.empty((B,), dtype=torch.int32, device="cuda"), torch.empty((B,), dtype=torch.int32, device="cuda")
    draft = torch.full((B, N, V), 1.0 / V, device="cuda")
    feat = torch.empty((B, N, H), dtype=dt, device="cuda")
    out = torch.empty((B, N, Hq, D), dtype=dt, device="cuda")

    def history_check(q_rot, kt, vt, par, got):
        longest = max(h.shape[0] for h in hist_k)
        pool_k = torch.zeros((B, Hkv, longest, D), dtype=dt)
        pool_v = torch.zeros_like(pool_k)
        for b in range(B):
            n = hist_k[b].shape[0]
            pool_k[b, :, :n], pool_v[b, :, :n] = hist_k[b].transpose(0, 1), hist_v[b].transpose(0, 1)
        want, bound = ref.attention(q_rot.cpu(), pool_k, pool_v, torch.arange(B)[:, None],
                                    [h.shape[0] for h in hist_k], kt.cpu(), vt.cpu(), par, D ** -0.5, dtype)
        assert ((got.double().cpu() - want).abs() <= bound).all()

    accepted = 0
    for step in range(3):
        q, k, v, hidden = rand(M, Hq, D).cuda(), rand(M, Hkv, D).cuda(), rand(B, N, Hkv, D).cuda(), rand(M, H).cuda()
        pos_d = (lens.cpu()[:, None] + depth[None]).to(torch.int32).flatten().cuda()
        q_rot, k_rot = torch.empty_like(q), torch.empty_like(k)
        cuda_lib.rope_append(shape, None, q, k, None, pos_d, None, cs_d, None, None, None, q_rot, k_rot)
        q4, k4 = q_rot.view(B, N, Hq, D), k_rot.view(B, N, Hkv, D)
        cuda_lib.tree_attention_paged(shape, pages, q4, kp, vp, table_d, lens, prompt, k4, v, parents.cuda(), out, ws)
        cuda_lib.quantize_rows(hidden, x8, xs)
        cuda_lib.lm_head_logits_scaled(x8, xs, w8, wscale, logits)
        # tokens: the greedy choice of the parent for nodes 2 and 5, so that they are accepted
        best = logits.argmax(dim=1).view(B, N).cpu()
        tokens = torch.full((B, N), -1, dtype=torch.int32)
        tokens[:, :] = (best[:, :1] + 1) % V
        tokens[0, 2], tokens[0, 5] = best[0, 0], best[0, 2]
        if step:
            tokens[1, 1] = best[1, 0]
        cuda_lib.tree_accept(shape, logits, draft, tokens.cuda(), parents.cuda(), 0.0, 0, 0, acc, alen, nxt)
        cuda_lib.commit_accepted_paged(shape, pages, kp, vp, table_d, lens, k4, v, hidden, parents.cuda(), acc, alen,
                                       new_lens, feat)
        torch.cuda.synchronize()
        history_check(q4, k4, v, parents, out)
        rows, bound = ref.logits_scaled(x8.cpu(), xs.cpu(), w8.cpu(), wscale.cpu())
        assert ((logits.double().cpu() - rows).abs() <= bound).all()
        for b in range(B):
            path = [0] + acc[b, :int(alen[b])].tolist()
            accepted += len(path) - 1
            hist_k[b] = torch.cat([hist_k[b], k4[b, path].cpu()])
            hist_v[b] = torch.cat([hist_v[b], v[b, path].cpu()])
            assert torch.equal(feat[b, :len(path)], hidden.view(B, N, H)[b, path])
            assert int(new_lens[b]) == hist_k[b].shape[0]
        lens, new_lens = new_lens, lens
    assert accepted >= 6
    # decoding of single tokens, each appended in the same call that rotates it
    q, k, v = rand(B, Hq, D).cuda(), rand(B, Hkv, D).cuda(), rand(B, Hkv, D).cuda()
    q_rot, k_rot = torch.empty_like(q), torch.empty_like(k)
    cuda_lib.rope_append(one, pages, q, k, v, lens, torch.arange(B, dtype=torch.int32).cuda(), cs_d, kp, vp, table_d,
                         q_rot, k_rot)
    root = torch.full((B, 1), -1, dtype=torch.int32)
    got = torch.empty((B, 1, Hq, D), dtype=dt, device="cuda")
    cuda_lib.tree_attention_paged(one, pages, q_rot[:, None], kp, vp, table_d, lens, prompt, k_rot[:, None], v[:, None],
                                  root.cuda(), got, ws)
    torch.cuda.synchronize()
    history_check(q_rot[:, None], k_rot[:, None], v[:, None], root, got)
