"""Host-side checks of include/ssm2d_ops.h that need no GPU: every declared
function is exported and bound, and arguments are refused with their documented
status before any call of the HIP runtime (pointers here are never read)."""
import ctypes
import inspect
import os

import pytest

import selective_state_space_ssm2d_amd as pkg

torch = pytest.importorskip("torch")
from selective_state_space_ssm2d_amd import ops  # noqa: E402

HEADER = os.path.join(os.path.dirname(pkg.HEADER_PATH), "ssm2d_ops.h")
FAKE = 0x10000
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(pkg.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()


def test_exports_and_bindings():
    names = pkg.exported_names(HEADER)
    assert len(names) == 12 and set(names) == {n + s for n in ops._SIGNATURES for s in ("", "_bf16")}
    lib = pkg.load_library()
    for name in names:
        assert hasattr(lib, name), name
    for name in ops.__all__:
        assert getattr(pkg, name) is getattr(ops, name) and name in pkg.__all__
        assert inspect.getdoc(getattr(pkg, name)), name


def test_constants_match_the_header():
    text = open(HEADER).read()
    for name, value in (("LN_MAX_N", ops.LN_MAX_N), ("ROPE_MAX_AXES", ops.ROPE_MAX_AXES), ("ROPE_MAX_D", ops.ROPE_MAX_D),
                        ("DELTA_MAX_DK", ops.DELTA_MAX_DK), ("DELTA_MAX_DV", ops.DELTA_MAX_DV)):
        assert f"#define SSM2D_{name} {value}\n" in text
    assert "SSM2D_ROPE_INTERLEAVED 1u" in text and "SSM2D_ROPE_INVERSE 2u" in text


# ------------------------------------------------------------------ layer norm

def _norm(dtype, sizes, ptrs=None, bwd=False):
    n = 8 if bwd else 6
    ptrs = [FAKE] * n if ptrs is None else ptrs
    fn = ops._entry("ssm2d_layer_norm_bwd" if bwd else "ssm2d_layer_norm_fwd", dtype)
    return fn(*ptrs, *sizes, *([8, 1, 8, 1] if bwd else [8, 1, 1e-5]), None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bwd", [False, True])
def test_norm(dtype, bwd):
    call = lambda sizes, ptrs=None: _norm(dtype, sizes, ptrs, bwd)  # noqa: E731
    for sizes in ((-1, 8, 1), (2, -8, 1), (2, 8, -1)):
        assert call(sizes) == pkg.ERR_BAD_DIM
    assert call((2, ops.LN_MAX_N + 1, 1)) == pkg.ERR_UNSUPPORTED
    assert call((1 << 40, 16384, 1)) == pkg.ERR_UNSUPPORTED
    none = [None] * (8 if bwd else 6)
    for sizes in ((0, 8, 1), (2, 0, 1), (2, 8, 0)):
        assert call(sizes, none) == pkg.OK
    size = 4 if dtype == torch.float32 else 2
    need, wide = ([0, 2, 3, 4, 5], [1, 2, 3, 6, 7]) if bwd else ([0, 3], [1, 2, 4, 5])
    for i in need:
        assert call((2, 8, 1), [FAKE if j != i else None for j in range(len(none))]) == pkg.ERR_NULLPTR
    for i in range(len(none)):
        off = 2 if i in wide else size // 2
        assert call((2, 8, 1), [FAKE + (off if j == i else 0) for j in range(len(none))]) == pkg.ERR_MISALIGNED


# ------------------------------------------------------------------ rotary positions

def _rope(dtype, ptrs=None, flags=0, sections=(2, 2), shape=None, **change):
    d = dict(batch=1, tokens=4, heads_q=2, heads_k=1, d=8, n_axes=len(sections))
    d.update(change)
    s = ops._RopeShape(q_stride=(64, 16, 8), k_stride=(32, 8, 8), sections=tuple(sections) + (0,) * (4 - len(sections)), pos_stride=(4, 0), **d)
    fn = ops._entry("ssm2d_rope", dtype)
    return fn(*([FAKE] * 6 if ptrs is None else ptrs), s if shape is None else shape[0], flags, None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope(dtype):
    for name in ("batch", "tokens", "heads_q", "heads_k", "d"):
        assert _rope(dtype, **{name: -1}) == pkg.ERR_BAD_DIM, name
    assert _rope(dtype, sections=(3, 2)) == pkg.ERR_BAD_DIM  # 10 dims of 8
    assert _rope(dtype, sections=(-1, 2)) == pkg.ERR_BAD_DIM
    assert _rope(dtype, n_axes=0) == pkg.ERR_UNSUPPORTED
    assert _rope(dtype, n_axes=5) == pkg.ERR_UNSUPPORTED
    assert _rope(dtype, d=ops.ROPE_MAX_D + 1) == pkg.ERR_UNSUPPORTED
    assert _rope(dtype, heads_q=65537) == pkg.ERR_UNSUPPORTED
    assert _rope(dtype, flags=4) == pkg.ERR_BAD_FLAGS
    assert _rope(dtype, shape=[None]) == pkg.ERR_NULLPTR
    for change in (dict(batch=0), dict(tokens=0), dict(heads_q=0, heads_k=0), dict(d=0, sections=(0,))):
        assert _rope(dtype, ptrs=[None] * 6, **change) == pkg.OK
    for i in range(6):
        assert _rope(dtype, ptrs=[FAKE if j != i else None for j in range(6)]) == pkg.ERR_NULLPTR, i
        off = 2 if i in (2, 3) else (2 if dtype == torch.float32 else 1)
        assert _rope(dtype, ptrs=[FAKE + (off if j == i else 0) for j in range(6)]) == pkg.ERR_MISALIGNED, i


# ------------------------------------------------------------------ gated delta rule

POINTERS = {"fwd": 9, "bwd": 15, "step": 7}
OPTIONAL = {"fwd": (5, 6, 8), "bwd": (5, 6, 8, 14), "step": ()}
FLOATS = {"fwd": (3, 4, 5, 6, 8), "bwd": (3, 4, 5, 8, 12, 13, 14), "step": (3, 4, 5)}  # aligned to 4 (cu_seqlens only when packed)


def _delta(kind, dtype, ptrs=None, shape=None, **change):
    d = dict(batch=2, tokens=100, n_seq=0, heads_qk=2, heads=4, d_k=16, d_v=16)
    d.update(change)
    st = lambda h, w: (d["tokens"] * h * w, h * w, w)  # noqa: E731
    strides = dict(q_stride=st(2, 16), k_stride=st(2, 16), v_stride=st(4, 16), do_stride=st(4, 16), g_stride=st(4, 1), beta_stride=st(4, 1))
    s = ops._DeltaShape(**{**strides, **d})
    fn = ops._entry("ssm2d_gated_delta_" + kind, dtype)
    return fn(*([FAKE] * POINTERS[kind] if ptrs is None else ptrs), s if shape is None else shape[0], 1.0, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", sorted(POINTERS))
def test_delta(kind, dtype):
    n = POINTERS[kind]
    for name in ("batch", "tokens", "heads_qk", "heads", "d_k", "d_v"):
        assert _delta(kind, dtype, **{name: -1}) == pkg.ERR_BAD_DIM, name
    assert _delta(kind, dtype, heads=5) == pkg.ERR_BAD_DIM
    assert _delta(kind, dtype, heads_qk=0) == pkg.ERR_BAD_DIM
    if kind == "step":
        assert _delta(kind, dtype, n_seq=1, batch=1) == pkg.ERR_BAD_FLAGS
    else:
        assert _delta(kind, dtype, n_seq=-1) == pkg.ERR_BAD_DIM
        assert _delta(kind, dtype, n_seq=3) == pkg.ERR_BAD_DIM  # (packed sequences in a batch of 2)
        packed = [FAKE if i != 6 else None for i in range(n)]
        assert _delta(kind, dtype, packed, n_seq=3, batch=1) == pkg.ERR_NULLPTR
    for change in (dict(d_k=129), dict(d_v=1025), dict(tokens=(1 << 31) - 64), dict(heads=1 << 15), dict(batch=1 << 22), dict(batch=1 << 24)):
        assert _delta(kind, dtype, **change) == pkg.ERR_UNSUPPORTED, change
    assert _delta(kind, dtype, shape=[None]) == pkg.ERR_NULLPTR
    for change in (dict(batch=0), dict(heads_qk=0, heads=0), dict(d_k=0, d_v=0, tokens=0)):
        assert _delta(kind, dtype, [None] * n, **change) == pkg.OK, change
    if kind != "bwd":  # outputs of no keys are zeros; those of no values are empty
        assert _delta(kind, dtype, [None] * n, d_k=0) == pkg.ERR_NULLPTR
        assert _delta(kind, dtype, [None] * n, d_v=0) == pkg.OK
    else:
        assert _delta(kind, dtype, [None] * n, d_k=0) == pkg.ERR_NULLPTR
        assert _delta(kind, dtype, [None] * n, d_v=0) == pkg.ERR_NULLPTR
    for i in range(n):
        if i not in OPTIONAL[kind]:
            assert _delta(kind, dtype, [FAKE if j != i else None for j in range(n)]) == pkg.ERR_NULLPTR, i
        if i == 6 and kind != "step":
            continue
        off = 2 if i in FLOATS[kind] or dtype == torch.float32 else 1
        assert _delta(kind, dtype, [FAKE + (off if j == i else 0) for j in range(n)]) == pkg.ERR_MISALIGNED, i


# ------------------------------------------------------------------ the binding

def test_binding_refuses_tensors_off_the_gpu():
    x, w = torch.zeros(2, 8), torch.ones(8)
    q, g = torch.zeros(1, 3, 2, 8), torch.zeros(1, 3, 2)
    pos = torch.zeros(1, 3, dtype=torch.int32)
    calls = [lambda: pkg.layer_norm_fwd(x, w), lambda: pkg.layer_norm_bwd(x, w, x[:, 0], x[:, 0], x),
             lambda: pkg.rope_fwd(q, None, pos, torch.zeros(4), (4,)), lambda: pkg.gated_delta_fwd(q, q, q, g, g),
             lambda: pkg.gated_delta_bwd(q, q, q, g, g, q), lambda: pkg.gated_delta_step(q, q, q, g, g, torch.zeros(1, 2, 8, 8))]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        pkg.layer_norm_fwd(x.double())


def test_norm_layout_of_empty_maps():
    """Maps without cells lie anyhow: their strides say nothing."""
    for shape in ((2, 3, 4, 0), (2, 3, 0, 4), (2, 3, 0, 0), (0, 3, 4, 4), (2, 0, 4, 4)):
        x = torch.empty(shape)
        b, n, cells, _, _ = ops._norm_layout(x, True)
        assert (b, n, cells) == (shape[0], shape[1], shape[2] * shape[3]), shape
    with pytest.raises(ValueError):
        ops._norm_layout(torch.empty(2, 3, 4, 5).transpose(2, 3), True)


def test_rope_sections_are_read_at_each_call():
    """Sections held in tensors that change are not answered from an earlier call; halves of a pair are refused."""
    sections = [torch.tensor(2), torch.tensor(3)]
    assert ops._sections(tuple(sections)) == ((2, 3), 5)
    sections[0].fill_(1)
    assert ops._sections(tuple(sections)) == ((1, 3), 4)
    with pytest.raises(TypeError):
        ops._sections((2.5, 1))


def test_norm_bwd_needs_the_statistics():
    x = torch.zeros(2, 8)
    for mean, rstd in ((None, x[:, 0]), (x[:, 0], None), (None, None)):
        with pytest.raises(ValueError, match="mean and rstd"):
            pkg.layer_norm_bwd(x, None, mean, rstd, x)
