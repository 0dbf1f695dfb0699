"""Host-side checks of include/ssm2d_block.h that need no GPU: every declared
function is exported and bound, and arguments are refused with their documented
status before any call of the HIP runtime (pointers here are never read)."""
import inspect
import os

import pytest

import selective_state_space_ssm2d_amd as pkg

torch = pytest.importorskip("torch")
from selective_state_space_ssm2d_amd import block  # noqa: E402

HEADER = os.path.join(os.path.dirname(pkg.HEADER_PATH), "ssm2d_block.h")
FAKE = 0x10000
DTYPES = [torch.float32, torch.bfloat16]
HUGE = 1 << 62


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(pkg.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()


def test_exports_and_bindings():
    names = set(pkg.exported_names(HEADER))
    both = {n + s for n in (*block._SIGNATURES, *block._WORKSPACES) for s in ("", "_bf16")} | set(block._PLAIN_WORKSPACES)
    assert names == both
    lib = pkg.load_library()
    for name in names:
        assert hasattr(lib, name), name
    for name in block.__all__:
        assert getattr(pkg, name) is getattr(block, name) and name in pkg.__all__
        assert inspect.getdoc(getattr(pkg, name)), name


def test_constants_match_the_header():
    text = open(HEADER).read()
    assert f"#define SSM2D_NORM_MAX_N {block.NORM_MAX_N}\n" in text
    for name in ("LINEAR_X_MAPS", "LINEAR_Y_MAPS", "NORM_ON", "NORM_GATE_SIGMOID", "NORM_GATE_FIRST", "NORM_RESIDUAL_F32", "RECUR_SIGMOID", "RECUR_MAPS",
                 "RECUR_REVERSE"):
        assert f"#define SSM2D_{name} {getattr(block, name)}u\n" in text
    for act, value in block.ACTS.items():
        assert f"#define SSM2D_ACT_{(act or 'none').upper()} {value}\n" in text


# ------------------------------------------------------------------ linear

def _linear(kind, dtype, ptrs=None, act=2, flags=0, shape=None, ws=FAKE, ws_bytes=HUGE, strides=None, **change):
    d = dict(batch=2, rows=10, n=8, k=16)
    d.update(change)
    st = dict(x_stride=(160, 16), r_stride=(80, 8), w_stride=16)
    st.update(strides or {})
    s = block._LinearShape(**d, **st)
    count = 7 if kind == "bwd" else 6
    fn = block._entry("ssm2d_linear_" + kind, dtype)
    return fn(*([FAKE] * count if ptrs is None else ptrs), s if shape is None else shape[0], act, flags, ws, ws_bytes, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_linear(kind, dtype):
    call = lambda **a: _linear(kind, dtype, **a)  # noqa: E731
    n = 7 if kind == "bwd" else 6
    for act in (-1, 4):
        assert call(act=act) == pkg.ERR_BAD_FLAGS
    assert call(flags=4) == pkg.ERR_BAD_FLAGS
    assert call(shape=[None]) == pkg.ERR_NULLPTR
    for name in ("batch", "rows", "n", "k"):
        assert call(**{name: -1}) == pkg.ERR_BAD_DIM, name
        assert call(**{name: 1 << 31}) == pkg.ERR_UNSUPPORTED, name
    assert call(batch=1 << 20, rows=1 << 20) == pkg.ERR_UNSUPPORTED
    assert call(strides=dict(w_stride=-16)) == pkg.ERR_BAD_DIM
    assert call(strides=dict(x_stride=(160, -16))) == pkg.ERR_BAD_DIM
    assert call(strides=dict(r_stride=(1 << 41, 8))) == pkg.ERR_UNSUPPORTED
    none = [None] * n
    if kind == "fwd":
        for change in (dict(batch=0), dict(rows=0), dict(n=0)):
            assert call(ptrs=none, ws=None, ws_bytes=0, **change) == pkg.OK
        need = (0, 1, 4)
    else:  # (outputs that are not given are not cleared)
        for change in (dict(batch=0), dict(rows=0), dict(n=0)):
            assert call(ptrs=none, ws=None, ws_bytes=0, **change) == pkg.OK
        assert call(ptrs=[FAKE] * 4 + [None] * 3) == pkg.OK  # nothing is wanted
        need = (0, 1, 2, 3)
    for i in need:
        assert call(ptrs=[FAKE if j != i else None for j in range(n)]) == pkg.ERR_NULLPTR, i
    f32 = (2,) if kind == "fwd" else (6,)
    for i in range(n):
        off = 2 if i in f32 or dtype == torch.float32 else 1
        assert call(ptrs=[FAKE + (off if j == i else 0) for j in range(n)]) == pkg.ERR_MISALIGNED, i
    assert call(ws=FAKE + 8) == pkg.ERR_MISALIGNED
    if kind == "bwd":
        assert call(ws=None) == pkg.ERR_NOMEM
        assert call(ws_bytes=2 * 10 * 8 * 2) == pkg.ERR_NOMEM
    else:  # a long sum of few outputs is split
        long = dict(batch=1, rows=4, n=64, k=1 << 16, strides=dict(x_stride=(0, 1 << 16), w_stride=1 << 16))
        assert call(**long, ws=None) == pkg.ERR_NOMEM
        assert call(**long, ws_bytes=16) == pkg.ERR_NOMEM


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_workspace(dtype):
    s = block._LinearShape(1, 4, 64, 1 << 16, (0, 1 << 16), (0, 64), 1 << 16)
    assert block._bytes("ssm2d_linear_fwd_workspace", dtype, s, 0) > 0
    assert block._bytes("ssm2d_linear_bwd_workspace", dtype, s, 2, 0) >= 4 * 64 * (4 if dtype == torch.float32 else 2)
    for bad in ((0, 4), (4, 0)):
        with pytest.raises(pkg.Ssm2dError):
            block._bytes("ssm2d_linear_bwd_workspace", dtype, s, *bad)
    with pytest.raises(pkg.Ssm2dError):
        block._bytes("ssm2d_linear_fwd_workspace", dtype, block._LinearShape(1, -4, 64, 8, (0, 8), (0, 64), 8), 0)
    big = block._LinearShape(1, 1 << 20, 4096, 4096, (0, 4096), (0, 4096), 4096)
    assert block._bytes("ssm2d_linear_fwd_workspace", dtype, big, 0) == 0


# ------------------------------------------------------------------ block norm

def _norm(kind, dtype, ptrs=None, flags=1, shape=None, ws=FAKE, ws_bytes=HUGE, **change):
    d = dict(rows=5, n=16, groups=2, x_stride=16, gate_stride=16, res_stride=16, dout_stride=16, dy_stride=16)
    d.update(change)
    s = block._NormShape(**d)
    s = s if shape is None else shape[0]
    fn = block._entry("ssm2d_block_norm_" + kind, dtype)
    if kind == "fwd":
        return fn(*([FAKE] * 8 if ptrs is None else ptrs), s, 1e-5, flags, None)
    return fn(*([FAKE] * 14 if ptrs is None else ptrs), s, 1e-5, flags, ws, ws_bytes, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_block_norm(kind, dtype):
    call = lambda **a: _norm(kind, dtype, **a)  # noqa: E731
    n = 8 if kind == "fwd" else 14
    assert call(flags=16) == pkg.ERR_BAD_FLAGS
    assert call(shape=[None]) == pkg.ERR_NULLPTR
    for change in (dict(rows=-1), dict(n=-16), dict(groups=0), dict(groups=-2), dict(groups=3), dict(x_stride=-1), dict(dy_stride=-16)):
        assert call(**change) == pkg.ERR_BAD_DIM, change
    assert call(n=block.NORM_MAX_N + 2) == pkg.ERR_UNSUPPORTED
    assert call(rows=1 << 48) == pkg.ERR_UNSUPPORTED
    for change in (dict(rows=0), dict(n=0)):
        assert call(ptrs=[None] * n, **change) == pkg.OK
    for i in (0, 6) if kind == "fwd" else (0,):
        assert call(ptrs=[FAKE if j != i else None for j in range(n)]) == pkg.ERR_NULLPTR, i
    f32 = (3, 4, 5) if kind == "fwd" else (3, 4, 5, 11, 12, 13)
    res = (2, 6) if kind == "fwd" else (2, 6, 10)
    for i in range(n):
        off = 2 if i in f32 or dtype == torch.float32 else 1
        assert call(ptrs=[FAKE + (off if j == i else 0) for j in range(n)]) == pkg.ERR_MISALIGNED, i
        if i in res:
            assert call(ptrs=[FAKE + (2 if j == i else 0) for j in range(n)], flags=1 | block.NORM_RESIDUAL_F32) == pkg.ERR_MISALIGNED, i
    if kind == "bwd":
        assert call(ws=FAKE + 8) == pkg.ERR_MISALIGNED
        assert call(ws=None) == pkg.ERR_NOMEM and call(ws_bytes=5 * 3 * 16 * 4 - 1) == pkg.ERR_NOMEM
        s = block._NormShape(5, 16, 2, 16, 16, 16, 16, 16)
        assert block._bytes("ssm2d_block_norm_bwd_workspace", dtype, s, 1) == 5 * 3 * 16 * 4


# ------------------------------------------------------------------ recurrence

def _rec(kind, dtype, ptrs=None, flags=0, shape=None, ws=FAKE, ws_bytes=HUGE, strides=(320, 16), **change):
    d = dict(batch=2, tokens=20, channels=16, n_seq=0)
    d.update(change)
    s = block._RecurrenceShape(x_stride=strides, g_stride=strides, dh_stride=strides, **d)
    fn = block._entry("ssm2d_recurrence_" + kind, dtype)
    return fn(*([FAKE] * (6 if kind == "fwd" else 9) if ptrs is None else ptrs), s if shape is None else shape[0], flags, ws, ws_bytes, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_recurrence(kind, dtype):
    call = lambda **a: _rec(kind, dtype, **a)  # noqa: E731
    n = 6 if kind == "fwd" else 9
    assert call(flags=8) == pkg.ERR_BAD_FLAGS
    for flag in (block.RECUR_MAPS, block.RECUR_REVERSE):
        assert call(flags=flag, n_seq=1, batch=1) == pkg.ERR_BAD_FLAGS
    assert call(shape=[None]) == pkg.ERR_NULLPTR
    for change in (dict(batch=-1), dict(tokens=-1), dict(channels=-1), dict(n_seq=-1), dict(n_seq=2), dict(strides=(-1, 16)), dict(strides=(320, -16))):
        assert call(**change) == pkg.ERR_BAD_DIM, change
    for change in (dict(batch=1 << 31), dict(tokens=1 << 31), dict(channels=1 << 31), dict(batch=1 << 20, channels=1 << 12)):
        assert call(**change) == pkg.ERR_UNSUPPORTED, change
    none = [None] * n
    for change in (dict(batch=0), dict(channels=0), dict(tokens=0)):
        assert call(ptrs=none, **change) == pkg.OK, change
    for i in (0, 1, 4) if kind == "fwd" else (0, 1, 4, 6, 7):
        assert call(ptrs=[FAKE if j != i else None for j in range(n)]) == pkg.ERR_NULLPTR, i
    assert call(ptrs=[FAKE if j != 3 else None for j in range(n)], n_seq=2, batch=1) == pkg.ERR_NULLPTR
    f32 = (2, 5) if kind == "fwd" else (2, 5, 8)
    for i in range(n):
        if i == 3:
            continue
        off = 2 if i in f32 or dtype == torch.float32 else 1
        assert call(ptrs=[FAKE + (off if j == i else 0) for j in range(n)]) == pkg.ERR_MISALIGNED, i
    assert call(ptrs=[FAKE + (2 if j == 3 else 0) for j in range(n)], n_seq=2, batch=1) == pkg.ERR_MISALIGNED
    long = dict(tokens=5000, strides=(80000, 16))
    assert call(**long, ws=FAKE + 8) == pkg.ERR_MISALIGNED
    assert call(**long, ws=None) == pkg.ERR_NOMEM and call(**long, ws_bytes=8) == pkg.ERR_NOMEM


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_recurrence_limits_are_the_workspaces_too(kind, dtype):
    """A shape has a workspace if the entry takes it, else the entry's status (here with no pointers: a shape that is taken lacks them)."""
    n = 6 if kind == "fwd" else 9
    for n_seq, channels in ((65535, 65537), (65536, 65535), (65536, 65536), (1 << 20, 1 << 12), (1 << 26, 1 << 11), (1 << 30, 1 << 10), (3, 5)):
        d = dict(batch=1, tokens=20, channels=channels, n_seq=n_seq)
        s = block._RecurrenceShape(x_stride=(0, channels), g_stride=(0, channels), dh_stride=(0, channels), **d)
        status = _rec(kind, dtype, ptrs=[None] * n, shape=[s])
        need = block._entry(f"ssm2d_recurrence_{kind}_workspace", dtype)(s, 0)
        assert status == (pkg.ERR_UNSUPPORTED if n_seq * channels > 2 ** 32 - 256 else pkg.ERR_NULLPTR), (n_seq, channels)
        assert need >= 0 if status == pkg.ERR_NULLPTR else need == -status, (n_seq, channels)


# ------------------------------------------------------------------ the binding

def test_binding_refuses_tensors_off_the_gpu():
    x, w = torch.zeros(2, 8), torch.zeros(4, 8)
    s = torch.zeros(1, 3, 8)
    for call in (lambda: pkg.linear_fwd(x, w), lambda: pkg.linear_bwd(x, w, torch.zeros(2, 4)), lambda: pkg.block_norm_fwd(x),
                 lambda: pkg.block_norm_bwd(x, x), lambda: pkg.recurrence_fwd(s, s), lambda: pkg.recurrence_bwd(s, s, s),
                 lambda: pkg.recurrence_step(x, x, x.float())):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: pkg.linear_fwd(x.double(), w.double()), lambda: pkg.block_norm_fwd(x.half()), lambda: pkg.recurrence_fwd(s.half(), s.half())):
        with pytest.raises(TypeError):
            call()
