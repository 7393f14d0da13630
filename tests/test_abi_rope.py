"""Host validation of the rotary and qk-norm calls: refused before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

import dynamic_sparse_attention_estimate_gb300 as pkg
from dynamic_sparse_attention_estimate_gb300 import RopeTable
from dynamic_sparse_attention_estimate_gb300.binding import RopeDims, ViewStrides

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from dynamic_sparse_attention_estimate_gb300.build import build
    build()
    return pkg.load_library()


@pytest.fixture(autouse=True)
def no_gpu():
    """Made-up device addresses are only passed where no launch could follow."""
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed where no GPU is visible")


def dims(**over):
    d = RopeDims(B=2, H=3, N=40, d=64, pairing=0, pos_batched=0, eps=1e-6)
    d.rot[:] = (24, 20, 20)
    d.len[:] = (4, 16, 16)
    for k, v in over.items():
        if k in ("rot", "len"):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


X, Y, POS, TAB = 0x100000, 0x900000, 0x2000000, 0x3000000


def rope(lib, d, x=X, xs=None, y=Y, ys=None, pos=POS, tab=TAB, fn="dsv_rope3d_fwd"):
    return getattr(lib, fn)(d, x, xs, pos, tab, y, ys, None)


@pytest.mark.parametrize("over,status,what", [
    (dict(B=0), INVALID, b"B, H, N"), (dict(H=0), INVALID, b"B, H, N"), (dict(N=0), INVALID, b"B, H, N"),
    (dict(N=-1), INVALID, b"B, H, N"), (dict(N=1 << 33), INVALID, b"int32"), (dict(N=1 << 30, H=4), INVALID, b"int32"),
    (dict(B=1, H=1, N=2 ** 31 - 64), INVALID, b"int32"),
    (dict(d=96), UNSUPPORTED, b"64 or 128"), (dict(pairing=2), INVALID, b"pairing"),
    (dict(rot=(3, 0, 0)), INVALID, b"even"), (dict(rot=(-2, 0, 0)), INVALID, b"even"),
    (dict(rot=(32, 32, 2)), INVALID, b"at most d"), (dict(rot=(66, 0, 0)), INVALID, b"rot"),
    (dict(len=(0, 4, 4)), INVALID, b"len"), (dict(len=(1 << 32, 4, 4)), INVALID, b"len"),
    (dict(len=(1 << 30, 4, 4)), INVALID, b"table"),
    (dict(pairing=1, rot=(4, 4, 4)), UNSUPPORTED, b"multiple of 16"),
    (dict(eps=-1.0), INVALID, b"eps"), (dict(eps=float("nan")), INVALID, b"eps"), (dict(eps=float("inf")), INVALID, b"eps"),
])
def test_bad_dims(lib, over, status, what):
    d = dims(**over)
    for fn in ("dsv_rope3d_fwd", "dsv_rope3d_bwd"):
        assert rope(lib, d, fn=fn) == status
        assert what in lib.dsv_last_error_message()
    assert lib.dsv_rope3d_table_bytes(d) == 0
    assert lib.dsv_qk_norm_rope_bwd_workspace(d) == 0
    assert lib.dsv_qk_norm_rope_fwd(d, X, X, None, None, None, None, POS, TAB, Y, 2 * Y, None, None) == status


def test_null_dims_and_pointers(lib):
    assert rope(lib, None) == INVALID
    d = dims()
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(tab=None)):
        assert rope(lib, d, **kw) == INVALID and b"NULL" in lib.dsv_last_error_message()
    for kw in (dict(x=X + 8), dict(y=Y + 2), dict(pos=POS + 4), dict(tab=TAB + 8)):
        assert rope(lib, d, **kw) == INVALID and b"aligned" in lib.dsv_last_error_message()


def test_table_sizes_and_theta(lib):
    d = dims()
    assert lib.dsv_rope3d_table_bytes(d) == 8 * (12 * 4 + 10 * 16 + 10 * 16)
    assert lib.dsv_rope3d_table_bytes(dims(rot=(0, 0, 0))) == 0
    th = (ctypes.c_double * 3)(1e4, 0.0, 1e4)
    assert lib.dsv_rope3d_table(d, th, TAB, None) == INVALID and b"theta[1]" in lib.dsv_last_error_message()
    assert lib.dsv_rope3d_table(d, None, TAB, None) == INVALID
    th[1] = float("inf")
    assert lib.dsv_rope3d_table(d, th, TAB, None) == INVALID
    th[1] = 1e4
    assert lib.dsv_rope3d_table(d, th, None, None) == INVALID
    # nothing rotated: nothing to fill
    assert lib.dsv_rope3d_table(dims(rot=(0, 0, 0)), None, None, None) == OK


def test_strides(lib):
    d = dims()
    for s in ((-8, 64, 192), (4, 2560, 64), (7680, 2560, 60), (1 << 41, 2560, 64)):
        assert rope(lib, d, xs=ViewStrides(*s)) == INVALID and b"strides" in lib.dsv_last_error_message()
    # elements of an output that fall on one another
    for s in ((7680, 2560, 0), (0, 2560, 64), (7680, 64, 64), (7680, 2552, 64), (7672, 2560, 64), (7680, 64, 184)):
        assert rope(lib, d, ys=ViewStrides(*s)) == INVALID and b"overlap" in lib.dsv_last_error_message()


def test_strides_that_span_too_much(lib):
    d = dims(B=1, H=1, N=2 ** 31 - 66)
    for s in (1 << 40, 1 << 39, 1 << 20):
        assert rope(lib, d, xs=ViewStrides(0, 0, s)) == INVALID and b"spans too much" in lib.dsv_last_error_message()


def test_outputs_over_inputs(lib):
    d = dims()
    size = 2 * 3 * 40 * 64 * 2
    # shifted by a row, one past, a different layout in place
    assert rope(lib, d, y=X + 128) == INVALID and b"overlaps" in lib.dsv_last_error_message()
    assert rope(lib, d, y=X - size + 16) == INVALID
    assert rope(lib, d, y=X, ys=ViewStrides(7680, 64, 192)) == INVALID
    args = lambda qo, ko, vo: (d, X, X + size, X + 2 * size, None, None, None, POS, TAB, qo, ko, vo, None)
    assert lib.dsv_qk_norm_rope_fwd(*args(X, Y, 2 * Y)) == INVALID
    assert lib.dsv_qk_norm_rope_fwd(*args(Y, Y, 2 * Y)) == INVALID
    assert lib.dsv_qk_norm_rope_fwd(*args(Y, Y + size - 16, 2 * Y)) == INVALID
    assert lib.dsv_qk_norm_rope_fwd(*args(Y, Y + size, X + 3 * size - 16)) == INVALID
    assert b"v_out overlaps v" in lib.dsv_last_error_message()


def bwd(lib, d, **over):
    size = 2 * 3 * 40 * 64 * 2
    a = dict(dq_out=X, dk_out=X + size, dv_out=X + 2 * size, q=X + 3 * size, k=X + 4 * size, strides=None, wq=TAB, wk=TAB,
             pos=POS, tab=TAB, dq=Y, dk=Y + size, dv=Y + 2 * size, ds=None, dwq=0x4000000, dwk=0x4001000, ws=0x5000000,
             nbytes=1 << 30)
    a.update(over)
    return lib.dsv_qk_norm_rope_bwd(d, *a.values(), None)


def test_backward_arguments(lib):
    d = dims()
    need = lib.dsv_qk_norm_rope_bwd_workspace(d)
    assert need >= 2 * 64 * 4
    for kw in (dict(dq_out=None), dict(dk_out=None), dict(q=None), dict(k=None), dict(dq=None), dict(dk=None)):
        assert bwd(lib, d, **kw) == INVALID and b"NULL" in lib.dsv_last_error_message()
    for kw in (dict(dv=None), dict(dv_out=None)):
        assert bwd(lib, d, **kw) == INVALID and b"both" in lib.dsv_last_error_message()
    for kw in (dict(wq=TAB + 2), dict(wk=TAB + 8), dict(dwq=0x4000004), dict(dwk=0x4000008)):
        assert bwd(lib, d, **kw) == INVALID and b"aligned" in lib.dsv_last_error_message()
    assert bwd(lib, d, ws=None) == WORKSPACE
    assert bwd(lib, d, ws=0x5000010) == WORKSPACE
    assert bwd(lib, d, nbytes=need - 1) == WORKSPACE
    assert bwd(lib, d, dk=Y) == INVALID and b"dk overlaps dq" in lib.dsv_last_error_message()
    assert bwd(lib, d, dq=X) == INVALID and b"overlaps" in lib.dsv_last_error_message()


def test_sums_and_workspace_over_other_tensors(lib):
    d = dims()
    size = 2 * 3 * 40 * 64 * 2
    ws = lib.dsv_qk_norm_rope_bwd_workspace(d)
    for over, what in ((dict(dwq=Y), b"dwq overlaps dq"), (dict(dwk=X + 5 * size - 16), b"dwk overlaps k"),
                       (dict(dwk=0x4000000), b"dwk overlaps dwq"), (dict(ws=Y + 2 * size & ~255), b"ws overlaps"),
                       (dict(ws=0x4001000, nbytes=ws), b"ws overlaps dwk"), (dict(dwq=0x5000000 + ws - 16), b"ws overlaps dwq")):
        assert bwd(lib, d, **over) == INVALID and what in lib.dsv_last_error_message(), over
    # without sums the workspace is not read; side by side is fine
    assert bwd(lib, d, dwq=None, dwk=None, ws=Y) not in (INVALID, WORKSPACE)
    assert bwd(lib, d, dwq=0x5000000 + ws, nbytes=ws) not in (INVALID, WORKSPACE)


def test_outputs_over_weights_positions_and_table(lib):
    """No output, sum or workspace may lie over a tensor that the same call reads: pos, table, wq, wk."""
    d = dims()
    N, f = d.N, d.d
    table, pos = lib.dsv_rope3d_table_bytes(d), 12 * N
    error = lib.dsv_last_error_message
    size = 2 * 3 * N * f * 2
    for fn in ("dsv_rope3d_fwd", "dsv_rope3d_bwd"):
        for kw, what in ((dict(pos=Y), b"pos"), (dict(pos=Y + size - 16), b"pos"), (dict(pos=Y - pos + 16 & ~15), b"pos"),
                         (dict(tab=Y), b"table"), (dict(tab=Y - table + 16), b"table"), (dict(tab=Y + size - 16), b"table")):
            assert rope(lib, d, fn=fn, **kw) == INVALID and b"overlaps " + what in error(), kw
        # in place too
        assert rope(lib, d, fn=fn, y=X, pos=X + 128) == INVALID and b"overlaps pos" in error()
        # side by side is fine
        assert rope(lib, d, fn=fn, pos=Y + size, tab=Y - table) not in (INVALID, WORKSPACE)
    # positions of every sample reach further
    b = dims(pos_batched=1)
    assert rope(lib, b, pos=Y - 2 * pos + 16) == INVALID and b"overlaps pos" in error()
    assert rope(lib, b, pos=Y - 2 * pos) not in (INVALID, WORKSPACE)

    def fwd(d=d, q_out=Y, k_out=Y + size, v_out=Y + 2 * size, wq=TAB, wk=TAB + 256, pos=POS, tab=TAB + 4096):
        return lib.dsv_qk_norm_rope_fwd(d, X, X + size, X + 2 * size, None, wq, wk, pos, tab, q_out, k_out, v_out, None)

    assert fwd() not in (INVALID, WORKSPACE)
    for i, name in enumerate((b"q_out", b"k_out", b"v_out")):
        at = Y + i * size
        for kw, what in ((dict(wq=at), b"wq"), (dict(wk=at + size - 16), b"wk"), (dict(pos=at + 256), b"pos"),
                         (dict(tab=at + 256), b"table")):
            assert fwd(**kw) == INVALID and name + b" overlaps " + what in error(), kw
    assert fwd(wq=Y - 2 * f) not in (INVALID, WORKSPACE)
    assert fwd(wq=Y - 2 * f + 16) == INVALID

    far, ws = 0x6000000, lib.dsv_qk_norm_rope_bwd_workspace(d)
    for out, start, end in (("dq", Y, Y + size), ("dk", Y + size, Y + 2 * size), ("dv", Y + 2 * size, Y + 3 * size),
                            ("dwq", 0x4000000, 0x4000000 + 4 * f), ("dwk", 0x4001000, 0x4001000 + 4 * f),
                            ("ws", 0x5000000, 0x5000000 + ws)):
        for name, key, span in (("wq", "wq", 2 * f), ("wk", "wk", 2 * f), ("pos", "pos", pos), ("table", "tab", table)):
            others = dict(wq=far, wk=far + 0x1000, pos=far + 0x2000, tab=far + 0x10000)
            for at in (start, end - 16) + ((start - span + 16,) if out not in ("dk", "dv") else ()):
                assert bwd(lib, d, **{**others, key: at}) == INVALID, (out, name, at)
                assert f"{out} overlaps {name}".encode() in error(), (out, name, at)
            if out not in ("dq", "dk"):   # (what follows those is the next output)
                assert bwd(lib, d, **{**others, key: end}) not in (INVALID, WORKSPACE), (out, name, error())
    # what a call does not read may lie anywhere: pos and table with nothing rotated, the workspace without sums
    still = dims(rot=(0, 0, 0))
    assert rope(lib, still, pos=Y, tab=Y) not in (INVALID, WORKSPACE)
    assert fwd(d=still, pos=Y, tab=Y) not in (INVALID, WORKSPACE)
    assert bwd(lib, d, dwq=None, dwk=None, ws=TAB) not in (INVALID, WORKSPACE)


def test_interleaved_outputs(lib):
    """The three views of a packed [B][N][3][H][d] gradient share a range but no element; shifted ones do."""
    d = dims()
    B, H, N, f = d.B, d.H, d.N, d.d
    packed = (ctypes.c_int64 * 9)(*(N * 3 * H * f, f, 3 * H * f) * 3)
    at = lambda i: Y + 2 * i * H * f
    # what follows the last check needs a device: the call gets there (no INVALID), or is refused for what is tested
    assert bwd(lib, d, ds=packed, dq=at(0), dk=at(1), dv=at(2)) not in (INVALID, WORKSPACE)
    assert bwd(lib, d, ds=packed, dq=at(2), dk=at(0), dv=at(1)) not in (INVALID, WORKSPACE)
    for k in (at(1) - 2 * f, at(0) + 16, at(1) + 2 * f, at(0) + 2 * 3 * H * f, at(3)):
        assert bwd(lib, d, ds=packed, dq=at(0), dk=k, dv=at(2)) == INVALID and b"overlaps" in lib.dsv_last_error_message()
    other = (ctypes.c_int64 * 9)(*(N * 3 * H * f, f, 3 * H * f), *(N * H * f, f, H * f), *(N * 3 * H * f, f, 3 * H * f))
    assert bwd(lib, d, ds=other, dq=at(0), dk=at(1), dv=at(2)) == INVALID


def test_overlapping_outputs_against_their_elements(lib):
    """Whether two outputs of one layout share an element, as the call sees it and by listing the elements."""
    import itertools
    import random
    rng = random.Random(4)
    seen = {True: 0, False: 0}
    for _ in range(300):
        B, H, N = (rng.randint(1, 3) for _ in range(3))
        d = dims(B=B, H=H, N=N, rot=(0, 0, 0))
        sizes, strides, extent = {"b": B, "h": H, "n": N}, {}, 64
        for a in rng.sample("bhn", 3):
            strides[a] = extent + 8 * rng.randint(0, 24)
            extent = strides[a] * (sizes[a] - 1) + extent
        shift = 8 * rng.randint(-40, 40)
        rows = [b * strides["b"] + h * strides["h"] + n * strides["n"]
                for b, h, n in itertools.product(range(B), range(H), range(N))]
        shared = bool({r + 8 * c for r in rows for c in range(8)} & {r + shift + 8 * c for r in rows for c in range(8)})
        view = (strides["b"], strides["h"], strides["n"])
        ds = (ctypes.c_int64 * 9)(*view * 3)
        far = 0x20000000
        status = bwd(lib, d, pos=None, tab=None, ds=ds, dq=Y, dk=Y + 2 * shift, dv=far, dq_out=far + 0x1000000,
                     dk_out=far + 0x2000000, dv_out=far + 0x3000000, q=far + 0x4000000, k=far + 0x5000000)
        assert (status == INVALID) == shared, (B, H, N, view, shift)
        seen[shared] += 1
    assert min(seen.values()) > 30


def test_python_refusals_without_a_gpu(lib):
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    pos = torch.zeros(8, 3, dtype=torch.int32)
    table = RopeTable(torch.zeros(64 * 8), (24, 20, 20), (1, 1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_rope3d_fwd(x, pos, table)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_qk_norm_rope_fwd(x, x, x, None, None, pos, table)
    with pytest.raises(TypeError):
        pkg.dsv_rope3d_bwd(None, pos, table)
    with pytest.raises(ValueError, match="three"):
        pkg.dsv_rope3d_table((24, 20), (4, 4), device="cpu")
    with pytest.raises(ValueError, match="pairing"):
        pkg.dsv_rope3d_table((24, 20, 20), (4, 4, 4), pairing="other", device="cpu")
    with pytest.raises(ValueError, match="theta"):
        pkg.dsv_rope3d_table((24, 20, 20), (4, 4, 4), theta=(1.0, 2.0), device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dsv_rope3d_table((24, 20, 20), (4, 4, 4), device="cpu")
