"""CPU checks of the 16-bit operators' calls: every refusal is a status code
returned before anything touches a GPU, empty calls succeed, workspace
queries are consistent, and the binding rejects unfit tensors."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import w4a4_quantized_gemm_smooth_b200 as S

vp = ctypes.c_void_p
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, NUMERIC = 0, 1, 2, 3, 4, 5
# aligned addresses that no refused call reads
A, B, C, D, E, F, G = (0x10000 * (i + 1) for i in range(7))


def linear(dtype=0, M=8, K=64, N=32, X=A, ldx=64, W=B, ldw=64, bias=None, R=None, ldr=0, epi=0, Y=C,
           ldy=32, P=None, ldp=0):
    return S.lib().svdq_linear16(dtype, M, K, N, X, ldx, W, ldw, bias, R, ldr, epi, Y, ldy, P, ldp, None)


def test_linear16_refusals():
    assert linear(M=0) == OK
    assert linear(dtype=2) == INVALID and linear(dtype=-1) == INVALID
    assert linear(epi=3) == INVALID and linear(epi=-1) == INVALID
    assert linear(M=-1) == SHAPE and linear(K=0) == SHAPE and linear(N=0) == SHAPE
    assert linear(ldx=56) == SHAPE and linear(ldw=56) == SHAPE and linear(ldy=24) == SHAPE
    assert linear(R=D, ldr=24) == SHAPE and linear(P=D, ldp=24) == SHAPE
    assert linear(M=0x7FFFFFFF) == UNSUPPORTED
    assert linear(K=0x7FFF8000, ldx=0x7FFF8000, ldw=0x7FFF8000) == UNSUPPORTED
    for k in ("X", "W", "Y"):
        assert linear(**{k: None}) == INVALID
        assert linear(**{k: 0x10008}) == ALIGN
    assert linear(P=C, ldp=32) == INVALID                       # P and Y are one array
    assert linear(R=D, ldr=32, P=D, ldp=32) == INVALID
    assert linear(R=C, ldr=40, ldy=32) == INVALID               # in place with another pitch
    assert linear(bias=0x10002) == ALIGN
    assert linear(R=0x10008, ldr=32) == ALIGN and linear(P=0x10008, ldp=32) == ALIGN
    assert linear(ldx=66) == ALIGN and linear(ldw=66) == ALIGN and linear(ldy=34) == ALIGN
    assert linear(R=D, ldr=34) == ALIGN and linear(P=D, ldp=34) == ALIGN


def linear_bwd(dtype=0, M=8, K=64, N=32, dY=A, lddy=32, X=B, ldx=64, W=C, ldw=64, P=D, ldp=32, epi=1,
               dX=E, lddx=64, dW=F, lddw=64, db=G, ws=0x100000, nbytes=1 << 30):
    return S.lib().svdq_linear16_backward(dtype, M, K, N, dY, lddy, X, ldx, W, ldw, P, ldp, epi, dX,
                                          lddx, dW, lddw, db, ws, nbytes, None)


def test_linear16_backward_refusals():
    assert linear_bwd(dX=None, dW=None, db=None) == OK          # nothing is asked for
    assert linear_bwd(dtype=2) == INVALID and linear_bwd(epi=3) == INVALID
    assert linear_bwd(M=-1) == SHAPE and linear_bwd(K=0) == SHAPE and linear_bwd(N=0) == SHAPE
    assert linear_bwd(lddy=24) == SHAPE and linear_bwd(ldx=56) == SHAPE and linear_bwd(ldw=56) == SHAPE
    assert linear_bwd(ldp=24) == SHAPE and linear_bwd(lddx=56) == SHAPE and linear_bwd(lddw=56) == SHAPE
    assert linear_bwd(N=0x7FFFFFFF, lddy=0x7FFFFFFF, ldp=0x7FFFFFFF) == UNSUPPORTED
    for k in ("dY", "X", "W", "P", "ws"):
        assert linear_bwd(**{k: None}) == INVALID
    for k in ("dY", "X", "W", "P", "dX", "dW"):
        assert linear_bwd(**{k: 0x10008}) == ALIGN
    assert linear_bwd(ws=0x100080) == ALIGN and linear_bwd(db=0x10001) == ALIGN
    need = S.svdq_linear16_backward_workspace(8, 64, 32, S.EPI_GELU)
    assert linear_bwd(nbytes=need - 1) == SHAPE
    assert S.svdq_linear16_backward_workspace(8, 64, 32, 3) == 0
    assert S.svdq_linear16_backward_workspace(0, 64, 32) == 0
    # dP of an activation is held in the workspace, rows padded to 16 bytes
    assert S.svdq_linear16_backward_workspace(1000, 64, 33, S.EPI_SILU) >= 1000 * 40 * 2


def test_linear16_backward_workspace_of_each_choice():
    """The query is enough for every choice of gradients, and a call asks for no
    more than it uses."""
    at = [i << 36 for i in range(1, 9)]
    dY, X, W, P, dX, dW, ws = at[:7]

    def need(M, K, N, epi, want_x, want_w):
        """The fewest bytes with which a call for db passes its check of the
        workspace.  db lies over dY, which is refused behind it: no launch."""
        k, n = (-(-v // 8) * 8 for v in (K, N))
        call = lambda size: S.lib().svdq_linear16_backward(
            0, M, K, N, dY, n, X, k, W, k, P, n, epi, dX if want_x else None, k, dW if want_w else None, k, dY, ws,
            size, None)
        lo, hi = 0, 1 << 34
        assert call(hi) == INVALID
        while lo < hi:
            mid = (lo + hi) // 2
            rc = call(mid)
            assert rc in (SHAPE, INVALID)
            lo, hi = (mid + 1, hi) if rc == SHAPE else (lo, mid)
        return lo

    for M in (1, 3, 8, 9, 32, 33, 1000):
        for K in (1, 64, 1152, 28672):
            for N in (1, 300, 8192):
                for epi in (S.EPI_NONE, S.EPI_GELU):
                    query = S.svdq_linear16_backward_workspace(M, K, N, epi)
                    for want in ((True, True), (True, False), (False, True), (False, False)):
                        n = need(M, K, N, epi, *want)
                        assert n <= query, (M, K, N, epi, want)
                        if not want[0] and M <= 8 and epi == S.EPI_NONE:
                            assert n == 0
                    # the bias's gradient alone is called without K
                    assert need(M, 1, N, epi, False, False) <= query


def test_form_sizes_reach_every_form():
    """Every instantiation of the tiled products (on pairs or clusters, tile
    width, splits, forward or gradients, one problem or two) is chosen for one
    of the sizes that the GPU tests run."""
    from test_gpu_ops16 import FORM_SIZES
    forms = {w: [S.svdq_debug_linear16_forms(*size, w) for size in sizes] for w, sizes in FORM_SIZES.items()}
    one = {w: {f[0] for f in fs if len(f) == 1} for w, fs in forms.items()}
    split = lambda widths: {(False, bn, s) for bn in widths for s in (1, 2, 4, 8) if bn // s >= 8}
    assert one[0] == split((32, 64, 128)) | {(True, bn, 1) for bn in (128, 192, 256)}
    grad = split((64, 128)) | {(True, bn, 1) for bn in (128, 256)}
    assert one[1] == grad and one[2] == grad
    # eight CTAs to a 128-wide tile of both: another form or two launches are always ahead of it
    assert one[3] == grad - {(False, 128, 8)}
    two = [f for f in forms[3] if len(f) == 2]
    assert len(two) >= 15 and {f[0] for f in two} | {f[1] for f in two} == grad
    # few rows take another way, and so does nothing else
    assert S.svdq_debug_linear16_forms(16, 64, 64) == [] and len(S.svdq_debug_linear16_forms(17, 64, 64)) == 1
    assert S.svdq_debug_linear16_forms(8, 64, 64, 3) == [] and len(S.svdq_debug_linear16_forms(9, 64, 64, 3)) == 1
    assert S.svdq_debug_linear16_forms(0, 64, 64) == [] and S.svdq_debug_linear16_forms(64, 64, 64, 4) == []
    assert S.lib().svdq_debug_linear16_forms(64, 64, 64, 0, None) == 0


def norm(dtype=0, pt=0, M=4, K=64, X=A, ldx=64, w=B, ldw=64, b=C, ldb=64, off=0.0, rpg=2, eps=1e-6,
         Y=D, ldy=64, mean=None, rstd=None):
    return S.lib().svdq_layer_norm(dtype, pt, M, K, X, ldx, w, ldw, b, ldb, off, rpg, eps, Y, ldy, mean,
                                   rstd, None)


def test_layer_norm_refusals():
    assert norm(M=0) == OK
    assert norm(dtype=3) == INVALID and norm(dtype=0, pt=1) == INVALID and norm(dtype=2, pt=0) == INVALID
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(eps=eps) == INVALID
    assert norm(off=math.nan) == INVALID
    assert norm(M=-1) == SHAPE and norm(K=0) == SHAPE and norm(rpg=-1) == SHAPE
    assert norm(ldx=56) == SHAPE and norm(ldy=56) == SHAPE and norm(ldw=56) == SHAPE and norm(ldb=56) == SHAPE
    assert norm(K=16385, ldx=16392, ldy=16392, ldw=16392, ldb=16392) == UNSUPPORTED
    assert norm(X=None) == INVALID and norm(Y=None) == INVALID
    assert norm(Y=A, ldy=72) == INVALID                          # in place with another pitch
    for k in ("X", "Y", "w", "b"):
        assert norm(**{k: 0x10004}) == ALIGN
    assert norm(ldx=66) == ALIGN and norm(ldy=66) == ALIGN and norm(ldw=66) == ALIGN and norm(ldb=66) == ALIGN
    assert norm(mean=0x10002) == ALIGN and norm(rstd=0x10001) == ALIGN


def norm_bwd(dtype=0, pt=2, M=4096, K=64, dY=A, lddy=64, X=B, ldx=64, mean=C, rstd=C, w=D, ldw=64, off=0.0,
             rpg=0, dX=E, lddx=64, dw=F, lddw=64, db=G, lddb=64, ws=0x100000, nbytes=1 << 30):
    return S.lib().svdq_layer_norm_backward(dtype, pt, M, K, dY, lddy, X, ldx, mean, rstd, w, ldw, off, rpg,
                                            dX, lddx, dw, lddw, db, lddb, ws, nbytes, None)


def test_layer_norm_backward_refusals():
    assert norm_bwd(dX=None, dw=None, db=None) == OK
    assert norm_bwd(M=0, rpg=2) == OK                            # no group, nothing to write
    assert norm_bwd(dtype=0, pt=1) == INVALID and norm_bwd(off=math.inf) == INVALID
    assert norm_bwd(M=-1) == SHAPE and norm_bwd(K=0) == SHAPE and norm_bwd(rpg=-1) == SHAPE
    for k in ("lddy", "ldx", "ldw", "lddx", "lddw", "lddb"):
        assert norm_bwd(**{k: 56}) == SHAPE
    assert norm_bwd(K=16385, **{k: 16392 for k in ("lddy", "ldx", "ldw", "lddx", "lddw", "lddb")}) == UNSUPPORTED
    for k in ("dY", "X", "mean", "rstd", "ws"):
        assert norm_bwd(**{k: None}) == INVALID
    assert norm_bwd(dX=A, lddx=72) == INVALID and norm_bwd(dX=B, lddx=72) == INVALID
    for k in ("dY", "X", "w", "dX", "dw", "db"):
        assert norm_bwd(**{k: 0x10004}) == ALIGN
    assert norm_bwd(ws=0x100010) == ALIGN and norm_bwd(mean=0x10002) == ALIGN
    need = S.svdq_layer_norm_backward_workspace(4096, 64, 0)
    assert need > 0 and norm_bwd(nbytes=need - 1) == SHAPE
    assert S.svdq_layer_norm_backward_workspace(4, 64, 1) == 0   # one row per group: no partial sums
    assert S.svdq_layer_norm_backward_workspace(4, 16385, 1) == 0


def plan(pairs=(8, 28, 28), freq=None, pairing=0, n=None):
    pp = np.asarray(pairs, np.int32)
    fr = np.asarray(np.ones(max(int(pp.clip(0).sum()), 1)) if freq is None else freq, np.float64)
    h = vp()
    rc = S.lib().svdq_rope_create(len(pp) if n is None else n, pp.ctypes.data_as(vp), fr.ctypes.data_as(vp),
                                  pairing, ctypes.byref(h))
    assert (rc == OK) == bool(h.value)
    return rc, h


def test_rope_plan_refusals():
    assert plan(n=0)[0] == INVALID and plan((1,) * 5)[0] == INVALID and plan(pairing=2)[0] == INVALID
    assert plan((0, 0))[0] == SHAPE and plan((-1, 3))[0] == SHAPE and plan((100, 29))[0] == SHAPE
    for f in (math.nan, math.inf, 2.0 ** 20, -2.0 ** 20):
        assert plan((1,), [f])[0] == NUMERIC
    assert S.lib().svdq_rope_create(1, None, None, 0, ctypes.byref(vp())) == INVALID
    for f in (0.0, -1.0, 1.0, 2 * math.pi, 1e-30):
        rc, h = plan((1,), [f])
        assert rc == OK
        S.lib().svdq_rope_free(h)
    S.lib().svdq_rope_free(None)


def test_rope_refusals():
    _, h = plan()

    def rope(dtype=0, T=4, H=2, D=128, pos=A, rows=4, ldp=3, X=B, xt=256, xh=128, Y=C, yt=256, yh=128, p=h):
        return S.lib().svdq_rope(p, dtype, T, H, D, pos, rows, ldp, X, xt, xh, Y, yt, yh, 0, None)

    assert rope(T=0) == OK and rope(H=0) == OK
    assert rope(p=None) == INVALID and rope(dtype=3) == INVALID
    assert rope(T=-1) == SHAPE and rope(H=-1) == SHAPE and rope(rows=0) == SHAPE and rope(ldp=2) == SHAPE
    assert rope(D=126) == SHAPE and rope(D=129, yh=129) == SHAPE and rope(D=0) == SHAPE
    assert rope(xt=-1) == SHAPE and rope(xh=-1) == SHAPE and rope(yt=-1) == SHAPE and rope(yh=-1) == SHAPE
    assert rope(yh=64) == SHAPE and rope(yt=64) == SHAPE         # heads or tokens of Y overlap
    assert rope(yt=200) == SHAPE and rope(H=3, yt=256, yh=130) == SHAPE
    assert rope(T=1, yt=0, X=0x10001) == ALIGN and rope(H=1, yh=0, X=0x10001) == ALIGN   # a single one has no stride
    assert rope(yh=1000, yt=128, X=0x10001) == ALIGN             # tokens within a head
    assert rope(D=1026, yh=1026, yt=4000) == UNSUPPORTED and rope(H=65536) == UNSUPPORTED
    assert rope(pos=None) == INVALID and rope(X=None) == INVALID and rope(Y=None) == INVALID
    assert rope(X=B, Y=B, yt=512) == INVALID                     # in place with other strides
    assert rope(X=0x10001) == ALIGN and rope(Y=0x10001) == ALIGN and rope(pos=0x10002) == ALIGN
    assert rope(dtype=2, X=0x10002) == ALIGN
    S.lib().svdq_rope_free(h)


def test_rope_of_no_tokens_takes_no_positions():
    p = S.svdq_rope_create([2], [1.0, 0.5])
    call = lambda T, rows: S.lib().svdq_rope(p.handle, 0, T, 2, 8, None, rows, 1, None, 16, 8, None, 16, 8, 0, None)
    assert call(0, 0) == OK and call(0, 5) == OK and call(0, -1) == SHAPE and call(1, 0) == SHAPE


# an output that shares memory with another array of its call: blocks run in any
# order, so the result would depend on timing
def test_linear16_refuses_overlap():
    M, K, N = 8, 64, 32
    x, w, y = M * K * 2, N * K * 2, M * N * 2
    assert linear(Y=A) == INVALID and linear(Y=B) == INVALID             # Y is X, Y is W
    assert linear(Y=A + x - 16) == INVALID and linear(Y=B + w - 16) == INVALID and linear(Y=A - y + 16) == INVALID
    assert linear(bias=C) == INVALID and linear(bias=C + y - 16) == INVALID
    assert linear(R=C + 16, ldr=32) == INVALID and linear(R=C - 64, ldr=32) == INVALID   # not quite in place
    assert linear(P=C + y - 64, ldp=32) == INVALID
    for P in (A, B, A + x - 16):
        assert linear(P=P, ldp=32) == INVALID
    assert linear(P=D, ldp=32, R=D + y - 16, ldr=32) == INVALID
    assert linear(P=D, ldp=32, bias=D + 16) == INVALID
    assert linear(R=C, ldr=32, P=C + 16, ldp=32) == INVALID              # in place, the pre-activation over it
    assert linear(M=200, ldx=128, ldy=128, Y=A + 96) == INVALID          # columns 48 to 79 of X's rows of 64 in 128
    assert linear(M=20, Y=A) == INVALID and linear(M=3000, Y=A) == INVALID


def test_linear16_backward_refuses_overlap():
    for name, others in (("dX", "dY X W P"), ("dW", "dY X W P dX"), ("db", "dY X W P dX dW"), ("ws", "dY X W P dX dW db")):
        for other in others.split():
            at = dict(dY=A, X=B, W=C, P=D, dX=E, dW=F, db=G)[other]
            assert linear_bwd(**{name: at}) == INVALID, (name, other)
            assert linear_bwd(M=40, **{name: at}) == INVALID, (name, other)
    assert linear_bwd(dX=B + 8 * 64 * 2 - 16) == INVALID                 # the last bytes of X


def test_layer_norm_refuses_overlap():
    assert norm(Y=A + 16) == INVALID and norm(Y=A + 4 * 64 * 2 - 16) == INVALID
    assert norm(Y=B) == INVALID and norm(Y=C) == INVALID
    for k in ("mean", "rstd"):
        for at in (A, B, C, D, D + 4 * 64 * 2 - 4):
            assert norm(**{k: at}) == INVALID
    assert norm(mean=E, rstd=E) == INVALID and norm(mean=E, rstd=E + 12) == INVALID
    H = 0x10000000           # apart from the others: 4096 rows of 64 take 512 KB
    far = dict(dY=H, X=2 * H, mean=3 * H, rstd=4 * H, w=5 * H, dX=6 * H, dw=7 * H, db=8 * H, ws=9 * H)
    for name, others in (("dX", "mean rstd w"), ("dw", "dY X mean rstd w dX"), ("db", "dY X mean rstd w dX dw"),
                         ("ws", "dY X mean rstd w dX dw db")):
        for other in others.split():
            assert norm_bwd(**{**far, name: far[other]}) == INVALID, (name, other)
    assert norm_bwd(**{**far, "dX": H + 128}) == INVALID and norm_bwd(**{**far, "dX": 2 * H - 128}) == INVALID


def test_rope_refuses_overlap():
    _, h = plan()

    def rope(T=4, H=2, D=128, pos=A, rows=4, X=B, xt=256, xh=128, Y=C, yt=256, yh=128):
        return S.lib().svdq_rope(h, 0, T, H, D, pos, rows, 3, X, xt, xh, Y, yt, yh, 0, None)

    size = 4 * 256 * 2
    assert rope(Y=B + 2) == INVALID and rope(Y=B - size + 2) == INVALID and rope(Y=B + size - 2) == INVALID
    assert rope(Y=B + 256) == INVALID                                    # head 0 over head 1
    assert rope(Y=B + 512, xt=512, yt=512, yh=128, T=3, H=3) == INVALID  # rows of 512: the third head meets the next
    assert rope(xt=0, Y=B + 256) == INVALID and rope(xh=0, Y=B + 512) == INVALID    # broadcast inputs
    assert rope(xt=128, xh=512, Y=B) == INVALID                          # other strides, the same memory
    assert rope(Y=A - 256) == INVALID and rope(pos=C + size - 4) == INVALID
    S.lib().svdq_rope_free(h)


def test_binding_rejects_unfit_tensors():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.zeros((16, 8), dtype=torch.bfloat16)
    y = torch.zeros((4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        S.svdq_linear16(x, w, y)
    with pytest.raises(ValueError, match="CUDA"):
        S.svdq_layer_norm(x, x)
    with pytest.raises(ValueError, match="dtype"):
        S.svdq_layer_norm(x.double(), x.double())
    with pytest.raises(ValueError, match="frequency"):
        S.svdq_rope_create([2, 2], [1.0])
    p = S.svdq_rope_create([2, 2], S.rope_frequencies([2, 2]))
    with pytest.raises(ValueError):
        S.svdq_rope(p, torch.zeros((4, 2), dtype=torch.int64), torch.zeros(4, 1, 8), torch.zeros(4, 1, 8))
    with pytest.raises(ValueError):
        S.svdq_rope(p, torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 8), torch.zeros(4, 8))
    p.free()
    p.free()


def test_norm_layer_refuses_to_save_what_it_overwrites():
    """The check stands before the call, so it needs no GPU."""
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    norm = S.LayerNorm()
    with pytest.raises(ValueError, match="save=True"):
        norm.forward(x, out=x, save=True)
    with pytest.raises(ValueError, match="CUDA"):       # the call itself, which wants a GPU's tensors
        norm.forward(x, out=x)
    with pytest.raises(ValueError, match="save=True"):  # its own buffer, fed back
        norm.forward(norm.Y, save=True)
    with pytest.raises(RuntimeError):
        norm.backward(x)


def test_binding_module_is_named_for_its_interpreter(tmp_path, monkeypatch):
    """A module that another interpreter's build left is not taken for this one's."""
    import sysconfig
    from w4a4_quantized_gemm_smooth_b200 import build
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert suffix.count(".") == 2                       # .cpython-3xx-<platform>.so
    assert os.path.basename(build.FASTCALL) == "_svdq_fastcall" + suffix
    monkeypatch.setattr(S, "_fast", None)
    assert S._fastcall().__file__ == build.FASTCALL
    (tmp_path / "_svdq_fastcall.so").write_bytes(b"another one's")
    monkeypatch.setattr(S, "_fast", None)
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / ("_svdq_fastcall" + suffix)))
    with pytest.raises(RuntimeError, match="missing"):
        S._fastcall()


@pytest.mark.parametrize("how", ["no gcc", "no headers"])
def test_library_builds_without_the_binding_module(tmp_path, monkeypatch, capfd, how):
    """The quantised layers do not need the module: the build reports that it
    is missing, leaves no older one, and the operators raise when called."""
    from w4a4_quantized_gemm_smooth_b200 import build
    at = tmp_path / "_svdq_fastcall.so"
    at.write_bytes(b"an older build's")
    os.utime(at, (0, 0))
    monkeypatch.setattr(build, "FASTCALL", str(at))
    run = build.subprocess.run

    def without(cmd, **kw):
        if cmd[0] != "gcc":
            return run(cmd, **kw)
        if how == "no gcc":
            raise FileNotFoundError(2, "No such file or directory", "gcc")
        headers = build.sysconfig.get_paths()["include"]
        return run([str(tmp_path) if c == headers else c for c in cmd], **kw)

    monkeypatch.setattr(build.subprocess, "run", without)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not at.exists()
    assert "16-bit operators" in capfd.readouterr().err
    monkeypatch.setattr(S, "_fast", None)
    with pytest.raises(RuntimeError, match="missing"):
        S._fastcall()


def test_binding_does_without_torchs_private_functions(monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(S, "_fast", None)
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        S.svdq_layer_norm(x, x.clone())


def test_rope_frequencies():
    assert S.rope_frequencies([2, 4], 100.0) == pytest.approx(
        [1.0, 0.1, 1.0, 100.0 ** -0.25, 0.1, 100.0 ** -0.75], rel=1e-15)


def test_programmatic_kernels_load_coherently():
    """Kernels that are resident while the one before them still writes (they
    call grid_wait) make no non-coherent load, nor let the compiler choose one
    through __restrict__."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(S.__file__), "csrc")
    shared = ("elem.cuh", "gemm16.cuh")
    seen = 0
    for path in sorted(glob.glob(os.path.join(csrc, "*.cu")) + glob.glob(os.path.join(csrc, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        if "grid_wait()" not in text and os.path.basename(path) not in shared:
            continue
        seen += 1
        found = re.findall(r"__ldg\b|__restrict__|\bld\.global\S*\.nc\b", text)
        assert not found, f"{os.path.basename(path)}: {found}"
    assert seen >= 8
