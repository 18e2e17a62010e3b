"""The paged-cache and e4m3 entry points reject bad arguments with a status before any CUDA
call (nothing here launches work)."""
import ctypes
import os
import re

import pytest
import torch

from tests import paged_ref as ref
from tree_verify_b200 import binding
from tree_verify_b200.build import build

FAKE = 1 << 24  # aligned fake device address; never dereferenced on these paths
INVALID, UNSUPPORTED, TOO_SMALL = (binding.EAGLE_ERR_INVALID_ARGUMENT, binding.EAGLE_ERR_UNSUPPORTED,
                                   binding.EAGLE_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def _shape(**kw):
    base = dict(batch=2, num_nodes=13, num_q_heads=8, num_kv_heads=2, head_dim=128, max_prefix_len=500,
                hidden=512, vocab=1000, dtype="bf16")
    base.update(kw)
    return binding.make_shape(**base)


def _pages(num=64, size=16, width=32):
    return binding.make_pages(num, size, width)


BAD_PAGES = [dict(num=0), dict(size=8), dict(size=48), dict(size=512), dict(size=0), dict(width=0),
             dict(size=256, width=1 << 23)]


# ------------------------------------------------------------------ attention

def _attend(lib, s=None, pg=None, shared=0, ptrs=None, ws=FAKE, ws_bytes=1 << 40):
    s, pg = s or _shape(), pg or _pages()
    # q, k_pages, v_pages, page_table, prefix_lens, (shared), k_tree, v_tree, parents, out
    p = ptrs or [FAKE] * 9
    return lib.eagle_tree_attention_paged(ctypes.byref(s), ctypes.byref(pg), *p[:5], shared, *p[5:], ws, ws_bytes,
                                          None)


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_attention_bad_pages(lib, bad):
    assert _attend(lib, pg=_pages(**bad)) == INVALID
    assert binding.paged_workspace_bytes(_shape(), _pages(**bad), 0) == 0


@pytest.mark.parametrize("bad", [dict(num_nodes=0), dict(num_nodes=65), dict(batch=0), dict(head_dim=96),
                                 dict(num_q_heads=6, num_kv_heads=4), dict(max_prefix_len=0), dict(dtype=7)])
def test_attention_bad_shapes(lib, bad):
    assert _attend(lib, s=_shape(**bad)) == INVALID


def test_attention_bad_lengths_pointers_and_workspace(lib):
    assert _attend(lib, shared=-1) == INVALID
    assert _attend(lib, shared=501) == INVALID                              # past max_prefix_len
    assert _attend(lib, s=_shape(max_prefix_len=513)) == INVALID            # past the table
    for i in range(9):
        p = [FAKE] * 9
        p[i] = None
        assert _attend(lib, ptrs=p) == INVALID, i
    for i in (0, 1, 2, 5, 6, 8):                                            # 16-byte operands
        p = [FAKE] * 9
        p[i] = FAKE + 8
        assert _attend(lib, ptrs=p) == INVALID, i
    assert lib.eagle_tree_attention_paged(None, ctypes.byref(_pages()), *([FAKE] * 5), 0, *([FAKE] * 4), FAKE,
                                          1 << 40, None) == INVALID
    assert lib.eagle_tree_attention_paged(ctypes.byref(_shape()), None, *([FAKE] * 5), 0, *([FAKE] * 4), FAKE,
                                          1 << 40, None) == INVALID
    assert _attend(lib, s=_shape(num_q_heads=258, num_kv_heads=2)) == UNSUPPORTED
    assert _attend(lib, s=_shape(batch=40000, num_q_heads=2)) == UNSUPPORTED


@pytest.mark.parametrize("shared", [0, 100, 500])
def test_attention_workspace(lib, shared):
    need = binding.paged_workspace_bytes(_shape(), _pages(), shared)
    assert need % 256 == 0
    if need:
        assert _attend(lib, shared=shared, ws_bytes=need - 1) == TOO_SMALL
        assert _attend(lib, shared=shared, ws=FAKE + 16, ws_bytes=need) == INVALID
        assert _attend(lib, shared=shared, ws=None, ws_bytes=need) == INVALID
    assert binding.paged_workspace_bytes(_shape(num_nodes=65), _pages(), 0) == 0
    assert binding.paged_workspace_bytes(_shape(), _pages(), 501) == 0


def test_attention_overlaps_and_longest_cache(lib):
    p = [FAKE + (i << 20) for i in range(9)]
    rows = 2 * 13 * 128 * 2
    for i, n in ((0, rows * 8), (5, rows * 2), (6, rows * 2)):              # q, k_tree, v_tree
        for at in (0, n - 16, 16 - rows * 8):
            x = list(p)
            x[8] = x[i] + at
            assert _attend(lib, ptrs=x) == INVALID, (i, at)
    wide = dict(size=256, width=(1 << 23) - 1)
    assert binding.paged_workspace_bytes(_shape(max_prefix_len=(1 << 31) - 513), _pages(**wide), 0) > 0
    assert binding.paged_workspace_bytes(_shape(max_prefix_len=(1 << 31) - 512), _pages(**wide), 0) == 0


@pytest.mark.parametrize("dtype,esize", [("bf16", 2), ("f32", 4)])
def test_attention_out_apart_from_the_cache_and_the_indices(lib, dtype, esize):
    out_bytes = 2 * 13 * 8 * 128 * esize
    # k_pages, v_pages, page_table, prefix_lens, parents of the default sizes
    for i, n in ((1, 64 * 2 * 16 * 128 * esize), (2, 64 * 2 * 16 * 128 * esize), (3, 2 * 32 * 4), (4, 2 * 4),
                 (7, 2 * 13 * 4)):
        for at in (0, (n - 1) // 16 * 16, 16 - out_bytes):
            p = [FAKE + (j << 22) for j in range(9)]
            p[8] = p[i] + at
            assert _attend(lib, s=_shape(dtype=dtype), ptrs=p, ws=FAKE + (9 << 22)) == INVALID, (i, at)


# ------------------------------------------------------------------ append

def _append(lib, s=None, pg=None, rope=(600, 64, 0), rows=7, **kw):
    s, pg = s or _shape(), pg or _pages()
    r = binding.Rope(*rope)
    qw, kw_ = s.num_q_heads * s.head_dim, s.num_kv_heads * s.head_dim
    big = 1 << 22
    a = dict(q=FAKE, qs=qw, k=FAKE + big, ks=kw_, v=FAKE + 2 * big, vs=kw_, pos=FAKE + 3 * big, seq=FAKE + 4 * big,
             cs=FAKE + 5 * big, kp=FAKE + 6 * big, vp=FAKE + 7 * big, pt=FAKE + 8 * big, qo=FAKE + 9 * big,
             ko=FAKE + 10 * big)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.eagle_rope_append(ctypes.byref(s), ctypes.byref(pg), ctypes.byref(r), rows, a["q"], a["qs"], a["k"],
                                 a["ks"], a["v"], a["vs"], a["pos"], a["seq"], a["cs"], a["kp"], a["vp"], a["pt"],
                                 a["qo"], a["ko"], None)


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_append_bad_pages(lib, bad):
    assert _append(lib, pg=_pages(**bad)) == INVALID


@pytest.mark.parametrize("rope", [(600, 8, 0), (600, 24, 0), (600, 144, 0), (600, -16, 0), (0, 64, 0), (600, 64, 2),
                                  (600, 64, -1)])
def test_append_bad_rope(lib, rope):
    assert _append(lib, rope=rope) == INVALID


def test_append_bad_arguments(lib):
    assert _append(lib, rows=-1) == INVALID
    assert _append(lib, rows=0, pos=None) == 0                     # nothing to do
    for name in ("q", "k", "v", "pos", "cs", "kp", "vp", "pt", "qo"):
        assert _append(lib, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "cs", "kp", "vp", "qo", "ko"):
        assert _append(lib, **{name: FAKE + 8}) == INVALID, name
    assert _append(lib, qs=1023) == INVALID                        # rows overlap
    assert _append(lib, ks=255) == INVALID
    assert _append(lib, vs=260) == INVALID                         # rows not 16-byte aligned
    assert _append(lib, q=None, qo=None, k=None, ko=None, seq=None) == INVALID  # nothing named
    assert _append(lib, seq=None, ko=None) == INVALID              # keys that go nowhere
    assert _append(lib, qs=2048, qo=FAKE) == INVALID               # in place, but not dense
    assert _append(lib, qo=FAKE + 1024) == INVALID                 # partial overlap
    assert _append(lib, ko=FAKE + (1 << 22) + 512) == INVALID
    assert _append(lib, qo=FAKE + (1 << 22)) == INVALID            # queries over the keys
    assert _append(lib, ko=FAKE + 2 * (1 << 22)) == INVALID        # keys over the values
    assert _append(lib, ko=FAKE + 9 * (1 << 22)) == INVALID        # keys over the rotated queries


def test_append_in_place_spares_only_the_operand_itself(lib):
    """An input that lies where the in-place operand does is read while that one is rotated."""
    q, k, v, kp, vp, qo = (FAKE + i * (1 << 22) for i in (0, 1, 2, 6, 7, 9))
    alone = dict(num_q_heads=2, num_kv_heads=2)
    assert _append(lib, v=k, ko=k) == INVALID                      # values = keys, keys in place
    assert _append(lib, s=_shape(**alone), k=q, qo=q) == INVALID   # keys = queries, queries in place
    assert _append(lib, s=_shape(**alone), v=q, qo=q) == INVALID   # values = queries
    assert _append(lib, k=q, ko=q, qo=qo) == INVALID               # queries over the keys, keys in place


@pytest.mark.parametrize("rows", [1, 7])
def test_append_outputs_apart_from_the_cache(lib, rows):
    s, pool = _shape(), 64 * 2 * 16 * 128 * 2                      # bytes of the default pools
    kp, vp = FAKE + 6 * (1 << 22), FAKE + 7 * (1 << 22)
    for name, heads in (("qo", 8), ("ko", 2)):
        for base in (kp, vp):
            for at in (0, pool - 16, 16 - rows * heads * 128 * 2):
                assert _append(lib, s=s, rows=rows, **{name: base + at}) == INVALID, (name, at)


# ------------------------------------------------------------------ commit

def _commit(lib, s=None, pg=None, ptrs=None):
    s, pg = s or _shape(), pg or _pages()
    # k_pages, v_pages, table, lens, k_tree, v_tree, hidden, parents, accepted, accept_len, new_lens, feat
    p = ptrs or [FAKE + (i << 16) for i in range(12)]
    return lib.eagle_commit_accepted_paged(ctypes.byref(s), ctypes.byref(pg), *p, None)


def test_commit_bad_arguments(lib):
    for bad in BAD_PAGES:
        assert _commit(lib, pg=_pages(**bad)) == INVALID
    assert _commit(lib, s=_shape(num_nodes=65)) == INVALID
    for i in range(12):
        p = [FAKE + (j << 16) for j in range(12)]
        p[i] = None
        assert _commit(lib, ptrs=p) == INVALID, i
    p = [FAKE + (j << 16) for j in range(12)]
    p[10] = p[3] + 4  # new_prefix_lens overlaps prefix_lens
    assert _commit(lib, ptrs=p) == INVALID
    p = [FAKE + (j << 16) for j in range(12)]
    p[11] = p[6] + 2 * 13 * 512 * 2 - 16  # feat overlaps hidden
    assert _commit(lib, ptrs=p) == INVALID


# ------------------------------------------------------------------ e4m3

@pytest.mark.parametrize("name", ["eagle_quantize_rows", "eagle_quantize_blocks"])
def test_quantize_bad_arguments(lib, name):
    f = getattr(lib, name)
    ok = (4, 256, 1, FAKE, FAKE, FAKE, None)
    for i, v in [(0, -1), (1, 0), (1, 8), (1, 200), (2, 2), (2, -1), (3, None), (4, None), (5, None), (3, FAKE + 8),
                 (4, FAKE + 8), (5, FAKE + 2)]:
        a = list(ok)
        a[i] = v
        assert f(*a) == INVALID, (i, v)
    assert f(0, 256, 1, None, None, None, None) == 0
    x, x8, sc = FAKE, FAKE + (1 << 16), FAKE + (2 << 16)
    for bad in ((x, x, sc), (x, x + 2032, sc), (x, x8, x8), (x, x8, x8 + 1008), (x, x8, x)):  # 4 x 256 bf16
        assert f(4, 256, 1, *bad, None) == INVALID, bad


def test_scaled_logits_bad_arguments(lib):
    f = lib.eagle_lm_head_logits_scaled
    ok = (4, 256, 100, FAKE, FAKE, FAKE, FAKE, FAKE, None)
    for i, v in [(0, -1), (1, 0), (1, 8), (1, 200), (2, 0), (3, None), (4, None), (5, None), (6, None), (7, None),
                 (3, FAKE + 8), (4, FAKE + 8), (5, FAKE + 8), (6, FAKE + 2), (7, FAKE + 2)]:
        a = list(ok)
        a[i] = v
        assert f(*a) == INVALID, (i, v)
    assert f(0, 256, 100, None, None, None, None, None, None) == 0
    p = [FAKE + (j << 20) for j in range(5)]
    for i, n in enumerate((4 * 256, 2 * 4 * 4, 100 * 256, 2 * 4)):          # logits over x, scales, w, scales
        for at in (0, n - 4, 4 - 4 * 100 * 4):
            assert f(4, 256, 100, *p[:4], p[i] + at, None) == INVALID, (i, at)
    assert f((1 << 24) + 1, 256, 100, FAKE, FAKE, FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert f(4, 256, 65536 * 128, FAKE, FAKE, FAKE, FAKE, FAKE, None) == UNSUPPORTED


def test_binding_checks_shapes():
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    x8 = torch.zeros((3, 256), dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        binding.quantize_rows(x, x8, torch.zeros((2, 3)))                       # rows not padded to 4
    with pytest.raises(ValueError):
        binding.quantize_blocks(x, x8, torch.zeros((2, 2)))
    with pytest.raises(ValueError):
        binding.lm_head_logits_scaled(x8, torch.zeros((2, 4)), x8, torch.zeros((1, 2)), torch.zeros((3, 4)))
    with pytest.raises(ValueError):
        binding.quantize_rows(x, x8, torch.zeros((2, 4)))                       # not device tensors


# ------------------------------------------------------------------ the plain forms themselves

def test_plain_block_scale_is_the_smallest():
    a = torch.tensor([0.0, 1.0, 448.0, 448.0000001, 447.9, 896.0, 1e-30, 3.0e38, 2.0 ** -149], dtype=torch.float64)
    s = ref.block_scale(a)
    assert (a <= 448 * s).all()
    assert ((a > 448 * s / 2) | (s == 2.0 ** -126)).all()


def test_plain_attention_sees_prefix_and_ancestors_only():
    torch.manual_seed(0)
    q = torch.randn(1, 3, 1, 64)
    kp, vp = torch.randn(4, 1, 16, 64), torch.randn(4, 1, 16, 64)
    kt, vt = torch.randn(1, 3, 1, 64), torch.randn(1, 3, 1, 64)
    table, parents = torch.tensor([[2, 0]]), torch.tensor([[-1, 0, 0]])
    out, _ = ref.attention(q, kp, vp, table, [17], kt, vt, parents, 0.125, "f32")
    keys = torch.cat([kp[2, 0], kp[0, 0, :1], kt[0, [0, 2], 0]]).double()
    vals = torch.cat([vp[2, 0], vp[0, 0, :1], vt[0, [0, 2], 0]]).double()
    want = torch.softmax(keys @ q[0, 2, 0].double() * 0.125, 0) @ vals
    assert torch.allclose(out[0, 2, 0], want, atol=1e-12)


# ------------------------------------------------------------------ waits that give up

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_verify_b200", "csrc")


def _kernel_body(name, kernel):
    """The kernel's body, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", text.index(kernel + "("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i], text
    raise AssertionError(f"{kernel} has no end")


@pytest.mark.parametrize("name,kernel", [("paged_attention_tc.cuh", "paged_attn_tc_kernel"),
                                         ("lm_head_scaled.cuh", "lm_head_scaled_kernel"),
                                         ("lm_head_scaled.cuh", "lm_head_scaled_rows_kernel")])
def test_a_warp_that_gave_up_leaves_nobody_at_a_barrier(name, kernel):
    """A warp whose bounded wait runs out leaves its loop alone and goes to the end of the kernel.
    Barriers that wait without a limit may so only stand where every thread passes once,
    outside all branches and loops; between warps of one role there are only bounded waits."""
    body, text = _kernel_body(name, kernel)
    assert not re.search(r"\bbar(rier)?(\.cta)?\.(sync|arrive|red)", text)
    depth, found = 0, 0
    for token in re.findall(r"[{}]|__syncthreads\w*\(|\bmbar_wait\(", body):
        depth += {"{": 1, "}": -1}.get(token, 0)
        if token.startswith("__syncthreads"):
            found += 1
            assert depth == 1, f"a block barrier at depth {depth}"
    assert found >= 2
