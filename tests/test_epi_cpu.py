"""CPU tests of the products with an epilogue, the layers grouped by expert and
the combination of rows: every refusal of the C ABI and of the binding, and the
argument checks under the address and undefined-behaviour sanitizers.  No test
here launches a kernel."""
import ctypes
import os
import shutil
import subprocess

import pytest

S = pytest.importorskip("w4a4_rank_corrected_amd")
from w4a4_rank_corrected_amd import _binding as B  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_rank_corrected_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")
FAKE = 0x10000      # never dereferenced: every call below is refused (or has nothing to do)
FAR = 0x40000000    # apart from FAKE by more than any tensor here
INVALID, UNSUPPORTED, ALIGN, WS = (B.SVDQ_ERR_INVALID_ARG, B.SVDQ_ERR_UNSUPPORTED, B.SVDQ_ERR_ALIGNMENT,
                                   B.SVDQ_ERR_WORKSPACE)


def _lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libsvdq.so not built")
    return B.lib()


def _layer(fmt="int4", **kw):
    d = dict(m=128, n=64, rank=8, group=64, smooth_inv=None, qw=FAKE, wscale=FAKE, l1=FAKE, l2=FAKE, bias=None, t=1.0,
             experts=4)
    d.update(kw)
    tail = (d["smooth_inv"], d["qw"], d["wscale"], d["l1"], d["l2"], d["bias"])
    if fmt == "int4":
        return B.svdq_layer(d["m"], d["n"], d["rank"], d["group"], *tail)
    if fmt == "w8a8":
        return B.svdq_w8a8_layer(d["m"], d["n"], d["rank"], *tail)
    if fmt == "fp4":
        return B.svdq_fp4_layer(d["m"], d["n"], d["rank"], d["t"], d["t"], *tail)
    return B.svdq_grouped_layer(d["experts"], d["m"], d["n"], d["rank"], d["group"], *tail)


def _epi(act=0, act_begin=0, gate_rows=0, ldr=0, ldy=0, gate=None, residual=None):
    return B.svdq_epilogue(act, act_begin, gate_rows, ldr, ldy, gate, residual)


BAD_EPILOGUES = [
    (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(act_begin=-1), INVALID), (dict(act_begin=65), INVALID),
    (dict(gate_rows=-1), INVALID),
    (dict(ldy=63), INVALID), (dict(ldy=-1), INVALID), (dict(ldy=B.SVDQ_MAX_DIM + 1), INVALID),
    (dict(ldr=63, residual=FAR), INVALID), (dict(ldr=B.SVDQ_MAX_DIM + 1, residual=FAR), INVALID),
    (dict(gate=FAR + 1), ALIGN), (dict(residual=FAR + 1), ALIGN),
    (dict(residual=FAKE + 2), INVALID),                      # overlaps y, but is not y
    (dict(residual=FAKE, ldr=128), INVALID),                 # y's address with another stride
    (dict(residual=FAKE + 2 * 63, ldr=128, ldy=128), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_EPILOGUES)
@pytest.mark.parametrize("fmt", ["int4", "w8a8", "fp4"])
def test_epilogue_refusals(fmt, kw, code):
    L = _lib()
    lay, epi = _layer(fmt), _epi(**kw)
    gemm = {"int4": L.svdq_gemm_w4a4_lowrank_up_epi, "w8a8": L.svdq_w8a8_gemm_lowrank_up_epi,
            "fp4": L.svdq_fp4_gemm_lowrank_up_epi}[fmt]
    linear = {"int4": L.svdq_linear_epi, "w8a8": L.svdq_w8a8_linear_epi, "fp4": L.svdq_fp4_linear_epi}[fmt]
    assert gemm(FAKE, FAKE, FAKE, ctypes.byref(lay), ctypes.byref(epi), 16, FAKE, 0, FAKE, 1 << 40, None) == code
    assert L.svdq_last_error()
    assert linear(FAKE, ctypes.byref(lay), ctypes.byref(epi), 16, FAKE, 0, FAKE, 1 << 40, None) == code


BAD_LAYERS = [(dict(m=100), UNSUPPORTED), (dict(n=0), INVALID), (dict(n=B.SVDQ_MAX_DIM + 1), UNSUPPORTED),
              (dict(rank=257), UNSUPPORTED), (dict(rank=-1), UNSUPPORTED), (dict(qw=None), INVALID),
              (dict(qw=FAKE + 8), ALIGN), (dict(wscale=None), INVALID), (dict(wscale=FAKE + 1), ALIGN),
              (dict(l2=None), INVALID), (dict(l2=FAKE + 1), ALIGN), (dict(bias=FAKE + 1), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_LAYERS)
def test_layer_refusals(kw, code):
    L = _lib()
    e = ctypes.byref(_epi(act=1))
    lay = _layer(**kw)
    assert L.svdq_gemm_w4a4_lowrank_up_epi(FAKE, FAKE, FAKE, ctypes.byref(lay), e, 16, FAKE, 0, FAKE, 1 << 40, None) == code
    assert L.svdq_linear_epi(FAKE, ctypes.byref(lay), e, 16, FAKE, 0, FAKE, 1 << 40, None) == code
    g = _layer("grouped", **kw)
    assert L.svdq_grouped_gemm_w4a4_lowrank_up(FAKE, FAKE, FAKE, FAKE, ctypes.byref(g), e, 16, FAKE, 0, None) == code
    assert L.svdq_grouped_linear(FAKE, 16, None, FAKE, ctypes.byref(g), e, 16, FAKE, 0, FAKE, 1 << 40, None) == code


def test_product_refusals():
    L = _lib()
    lay = ctypes.byref(_layer())
    f = L.svdq_gemm_w4a4_lowrank_up_epi
    for args, code in [((None, FAKE, FAKE, lay, None, 16, FAKE, 0, FAKE, 0, None), INVALID),
                       ((FAKE + 8, FAKE, FAKE, lay, None, 16, FAKE, 0, FAKE, 0, None), ALIGN),
                       ((FAKE, None, FAKE, lay, None, 16, FAKE, 0, FAKE, 0, None), INVALID),
                       ((FAKE, FAKE + 1, FAKE, lay, None, 16, FAKE, 0, FAKE, 0, None), ALIGN),
                       ((FAKE, FAKE, None, lay, None, 16, FAKE, 0, FAKE, 0, None), INVALID),
                       ((FAKE, FAKE, FAKE + 2, lay, None, 16, FAKE, 0, FAKE, 0, None), ALIGN),
                       ((FAKE, FAKE, FAKE, None, None, 16, FAKE, 0, FAKE, 0, None), INVALID),
                       ((FAKE, FAKE, FAKE, lay, None, -1, FAKE, 0, FAKE, 0, None), INVALID),
                       ((FAKE, FAKE, FAKE, lay, None, B.SVDQ_MAX_DIM + 1, FAKE, 0, FAKE, 0, None), UNSUPPORTED),
                       ((FAKE, FAKE, FAKE, lay, None, 16, None, 0, FAKE, 0, None), INVALID),
                       ((FAKE, FAKE, FAKE, lay, None, 16, FAKE, 2, FAKE, 0, None), INVALID),
                       ((FAKE, FAKE, FAKE, lay, None, 16, FAKE + 2, 1, FAKE, 0, None), ALIGN)]:
        assert f(*args) == code, args
    assert f(FAKE, FAKE, FAKE, lay, None, 0, None, 0, None, 0, None) == B.SVDQ_OK  # nothing to do
    wide = ctypes.byref(_layer(m=4096))
    need = L.svdq_gemm_epi_workspace_size(256, 64, 4096)
    assert need > 0 and L.svdq_gemm_epi_workspace_size(16, 64, 4096) == 0
    assert f(FAKE, FAKE, FAKE, wide, None, 256, FAKE, 0, FAKE, need - 1, None) == WS
    assert f(FAKE, FAKE, FAKE, wide, None, 256, FAKE, 0, None, need, None) == WS
    assert f(FAKE, FAKE, FAKE, wide, None, 256, FAKE, 0, FAKE + 8, need, None) == ALIGN
    lin = L.svdq_linear_epi
    need = L.svdq_linear_workspace_size(16, 128, 64, 8, 64)
    assert lin(FAKE, lay, None, 16, FAKE, 0, FAKE, need - 1, None) == WS
    assert lin(FAKE, lay, None, 16, FAKE, 0, FAKE + 16, need, None) == ALIGN
    assert lin(None, lay, None, 16, FAKE, 0, FAKE, need, None) == INVALID
    assert lin(FAKE + 2, lay, None, 16, FAKE, 0, FAKE, need, None) == ALIGN
    assert lin(FAKE, ctypes.byref(_layer(l1=None)), None, 16, FAKE, 0, FAKE, need, None) == INVALID
    assert lin(FAKE, ctypes.byref(_layer(smooth_inv=FAKE + 4)), None, 16, FAKE, 0, FAKE, need, None) == ALIGN
    assert L.svdq_w8a8_linear_epi(FAKE, ctypes.byref(_layer("w8a8", l1=None)), None, 16, FAKE, 0, FAKE, 1 << 40, None) == INVALID
    assert L.svdq_fp4_linear_epi(FAKE, ctypes.byref(_layer("fp4", t=0.3)), None, 16, FAKE, 0, FAKE, 1 << 40, None) == INVALID


def test_grouped_refusals():
    L = _lib()
    g = ctypes.byref(_layer("grouped"))
    q, p, lin = (L.svdq_grouped_quantize_act_lowrank_down, L.svdq_grouped_gemm_w4a4_lowrank_up, L.svdq_grouped_linear)
    for kw, code in [(dict(experts=0), INVALID), (dict(experts=1025), UNSUPPORTED), (dict(group=32), UNSUPPORTED)]:
        bad = ctypes.byref(_layer("grouped", **kw))
        assert q(FAKE, 16, None, FAKE, bad, 16, FAKE, FAKE, FAKE, None) == code
        assert p(FAKE, FAKE, FAKE, FAKE, bad, None, 16, FAKE, 0, None) == code
        assert lin(FAKE, 16, None, FAKE, bad, None, 16, FAKE, 0, FAKE, 1 << 40, None) == code
    for args, code in [((None, 16, None, FAKE, g, 16, FAKE, FAKE, FAKE, None), INVALID),
                       ((FAKE + 8, 16, None, FAKE, g, 16, FAKE, FAKE, FAKE, None), ALIGN),
                       ((FAKE, 16, None, None, g, 16, FAKE, FAKE, FAKE, None), INVALID),
                       ((FAKE, 16, None, FAKE + 2, g, 16, FAKE, FAKE, FAKE, None), ALIGN),
                       ((FAKE, 16, FAKE + 2, FAKE, g, 16, FAKE, FAKE, FAKE, None), ALIGN),
                       ((FAKE, 15, None, FAKE, g, 16, FAKE, FAKE, FAKE, None), INVALID),   # x shorter than b, no index
                       ((FAKE, 0, FAKE, FAKE, g, 16, FAKE, FAKE, FAKE, None), INVALID),
                       ((FAKE, B.SVDQ_MAX_DIM + 1, FAKE, FAKE, g, 16, FAKE, FAKE, FAKE, None), UNSUPPORTED),
                       ((FAKE, 16, None, FAKE, g, 16, None, FAKE, FAKE, None), INVALID),
                       ((FAKE, 16, None, FAKE, g, 16, FAKE, FAKE, None, None), INVALID),
                       ((FAKE, 16, None, FAKE, None, 16, FAKE, FAKE, FAKE, None), INVALID),
                       ((FAKE, 16, None, FAKE, g, -1, FAKE, FAKE, FAKE, None), INVALID)]:
        assert q(*args) == code, args
    for e in (_epi(gate=FAR), _epi(residual=FAR)):
        assert p(FAKE, FAKE, FAKE, FAKE, g, ctypes.byref(e), 16, FAKE, 0, None) == UNSUPPORTED
    for kw, code in BAD_EPILOGUES:
        if "gate" not in kw and "residual" not in kw:
            assert p(FAKE, FAKE, FAKE, FAKE, g, ctypes.byref(_epi(**kw)), 16, FAKE, 0, None) == code
    assert p(FAKE, FAKE, FAKE, None, g, None, 16, FAKE, 0, None) == INVALID
    assert p(FAKE, FAKE, None, FAKE, g, None, 16, FAKE, 0, None) == INVALID
    assert p(FAKE, FAKE, FAKE, FAKE, g, None, 16, None, 0, None) == INVALID
    huge = ctypes.byref(_layer("grouped", n=B.SVDQ_MAX_DIM, experts=1024))
    assert p(FAKE, FAKE, FAKE, FAKE, huge, None, B.SVDQ_MAX_DIM, FAKE, 0, None) == UNSUPPORTED
    need = L.svdq_grouped_linear_workspace_size(16, 4, 128, 64, 8)
    assert lin(FAKE, 16, None, FAKE, g, None, 16, FAKE, 0, FAKE, need - 1, None) == WS
    assert lin(FAKE, 16, None, FAKE, g, None, 16, FAKE, 0, FAKE + 16, need, None) == ALIGN
    assert lin(FAKE, 16, None, FAKE, ctypes.byref(_layer("grouped", l1=None)), None, 16, FAKE, 0, FAKE, need, None) == INVALID
    for f, args in ((q, (None, 0, None, None, g, 0, None, None, None, None)),
                    (p, (None, None, None, None, g, None, 0, None, 0, None)),
                    (lin, (None, 0, None, None, g, None, 0, None, 0, None, 0, None))):
        assert f(*args) == B.SVDQ_OK  # b == 0
    assert L.svdq_grouped_linear_workspace_size(0, 4, 128, 64, 8) == 0


def test_combine_refusals():
    L = _lib()
    f = L.svdq_combine_rows
    ok = dict(rows=FAR, R=8, n=64, dtype=0, index=FAR, weight=FAR, t=4, k=2, residual=None, y=FAKE)

    def st(**kw):
        d = dict(ok, **kw)
        return f(*(d[k] for k in ("rows", "R", "n", "dtype", "index", "weight", "t", "k", "residual", "y")), None)

    for kw, code in [(dict(R=-1), INVALID), (dict(n=0), INVALID), (dict(t=-1), INVALID), (dict(k=0), INVALID),
                     (dict(k=1025), UNSUPPORTED), (dict(R=B.SVDQ_MAX_DIM + 1), UNSUPPORTED),
                     (dict(t=B.SVDQ_MAX_DIM, n=B.SVDQ_MAX_DIM), UNSUPPORTED), (dict(dtype=2), INVALID),
                     (dict(rows=None), INVALID), (dict(index=None), INVALID), (dict(y=None), INVALID),
                     (dict(rows=FAR + 1), ALIGN), (dict(index=FAR + 2), ALIGN), (dict(weight=FAR + 1), ALIGN),
                     (dict(residual=FAR + 1), ALIGN), (dict(y=FAKE + 2, dtype=1), ALIGN),
                     (dict(rows=FAKE + 128), INVALID), (dict(residual=FAKE + 128), INVALID),
                     (dict(residual=FAKE - 128), INVALID)]:
        assert st(**kw) == code, kw
    assert st(t=0, rows=None, index=None, y=None) == B.SVDQ_OK


class _Fake:
    """A tensor's face for the binding's checks."""

    def __init__(self, shape, dtype, device="cuda:0", stride=None):
        import torch
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.is_cuda = True
        self._dense = tuple(int(__import__("math").prod(shape[i + 1:])) for i in range(len(shape)))
        self._stride = stride or self._dense

    def is_contiguous(self):
        return self._stride == self._dense

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._stride

    def data_ptr(self):
        return FAKE


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import types
    dev = torch.device("cuda:0")
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x = torch.zeros((4, 128), dtype=bf)
    lay = types.SimpleNamespace(m=128, n=64, rank=8, experts=4, qw=_Fake((2, 64, 32), torch.uint8))
    _lib()
    for f in (S.svdq_linear_epi, S.svdq_w8a8_linear_epi, S.svdq_fp4_linear_epi):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(x, lay)
        with pytest.raises(ValueError, match="channels"):
            f(_Fake((4, 64), bf), lay)
    for f, dt in ((S.svdq_gemm_w4a4_lowrank_up_epi, torch.uint8), (S.svdq_w8a8_gemm_lowrank_up_epi, torch.int8),
                  (S.svdq_fp4_gemm_lowrank_up_epi, torch.uint8)):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(torch.zeros((2, 4, 32), dtype=dt), None, None, lay)
    for f in (S.svdq_grouped_linear, S.svdq_grouped_quantize_act_lowrank_down):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(x, None, lay)
        with pytest.raises(ValueError, match="offsets has shape"):
            f(_Fake((4, 128), bf), _Fake((4,), i32), lay)
        with pytest.raises(ValueError, match="offsets has dtype"):
            f(_Fake((4, 128), bf), _Fake((5,), torch.int64), lay)
        with pytest.raises(ValueError, match="row_index has dtype"):
            f(_Fake((4, 128), bf), _Fake((5,), i32), lay, row_index=_Fake((9,), torch.int64))
        with pytest.raises(ValueError, match="row_index must be 1-D"):
            f(_Fake((4, 128), bf), _Fake((5,), i32), lay, row_index=_Fake((3, 3), i32))
        with pytest.raises(ValueError, match="channels"):
            f(_Fake((4, 64), bf), _Fake((5,), i32), lay)
    y = _Fake((4, 64), bf)
    for kw, what in [(dict(act="tanh"), "act must be"), (dict(act_begin=65), "act_begin"), (dict(act_begin=-1), "act_begin"),
                     (dict(gate=_Fake((4, 64), bf)), "gate has shape"), (dict(gate=_Fake((1, 64), f32)), "gate has dtype"),
                     (dict(gate=_Fake((1, 64), bf), gate_rows=-2), "gate_rows"),
                     (dict(residual=_Fake((4, 64), f32)), "residual has dtype"),
                     (dict(residual=_Fake((3, 64), bf)), "residual has shape"),
                     (dict(residual=_Fake((4, 64), bf, stride=(0, 1))), "row stride"),
                     (dict(residual=_Fake((4, 64), bf, stride=(1, 4))), "columns of residual"),
                     (dict(residual=_Fake((4, 64), bf, device="cuda:1")), "expected cuda:0"),
                     (dict(y=_Fake((4, 64), f32), out_dtype=bf), "y has dtype"),
                     (dict(y=_Fake((4, 64), bf, stride=(1 << 33, 1))), "row stride"),
                     (dict(out_dtype=torch.float16), "out_dtype")]:
        d = dict(y=y, out_dtype=None, act="none", act_begin=0)
        d.update(kw)
        with pytest.raises(ValueError, match=what):
            B._epilogue(4, 64, dev, **d)
    _, code, e = B._epilogue(5, 64, dev, y=_Fake((5, 64), f32, stride=(80, 1)), out_dtype=None, act="silu", act_begin=3,
                             gate=_Fake((3, 64), bf), gate_rows=2)
    assert (code, e.act, e.act_begin, e.gate_rows, e.ldy, e.ldr) == (1, 3, 3, 2, 80, 0)
    _, _, e = B._epilogue(5, 64, dev, y=_Fake((5, 64), f32), out_dtype=None, act="none", act_begin=0,
                          gate=_Fake((1, 64), bf), gate_rows=1 << 40)
    assert e.gate_rows == 5
    rows, idx = _Fake((8, 64), bf), _Fake((4, 2), i32)
    for args, kw, what in [((torch.zeros((8, 64)), None), {}, "GPU tensor"), ((_Fake((8, 64), torch.float16), idx), {}, "rows must"),
                           ((_Fake((8,), bf), idx), {}, "rows must"), ((rows, _Fake((4, 2), torch.int64)), {}, "index has dtype"),
                           ((rows, _Fake((4,), i32)), {}, "index must be 2-D"),
                           ((rows, idx), dict(weight=_Fake((4, 3), f32)), "weight has shape"),
                           ((rows, idx), dict(weight=_Fake((4, 2), bf)), "weight has dtype"),
                           ((rows, idx), dict(residual=_Fake((4, 64), f32)), "residual has dtype"),
                           ((rows, idx), dict(out_dtype=f32), "dtype of rows")]:
        with pytest.raises(ValueError, match=what):
            S.svdq_combine_rows(*args, **kw)
    with pytest.raises(ValueError, match="at least one"):
        S.GroupedDeviceLayer([])
    with pytest.raises(ValueError, match="different"):
        S.GroupedDeviceLayer([dict(m=64, n=8, rank=0), dict(m=64, n=16, rank=0)])
    with pytest.raises(ValueError, match="biases"):
        S.GroupedDeviceLayer([dict(m=64, n=8, rank=0)], biases=[])
    with pytest.raises(ValueError, match="GPU tensor"):
        S.GroupedDeviceLayer.from_tensors(1, 64, 8, 0, torch.zeros((1, 1, 8, 32), dtype=torch.uint8), None)
    with pytest.raises(ValueError, match="GPU tensor"):
        S.DeviceLayer8.from_tensors(64, 8, 0, torch.zeros((1, 8, 64), dtype=torch.int8), None)
    with pytest.raises(ValueError, match="wscale has shape"):
        S.DeviceLayerFp4.from_tensors(64, 8, 0, 1.0, 1.0, _Fake((1, 8, 32), torch.uint8), _Fake((1, 8), torch.uint8))


def test_argument_checks_under_address_and_ub_sanitizers(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "epi_sanitize")
    sources = [os.path.join(CSRC, f) for f in ("api.cpp", "epi_api.cpp", "prep.cpp", "bundle.cpp", "plan.cpp")] + \
              [os.path.join(NATIVE, f) for f in ("device_stubs.cpp", "epi_stubs.cpp", "epi_sanitize.cpp")]
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=undefined", "-ffp-contract=off", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    res = subprocess.run(["g++", *flags, *sources, "-o", exe, "-pthread"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1", TMPDIR=str(tmp_path)))
    out = run.stdout + run.stderr
    assert run.returncode == 0 and "epi sanitize ok" in run.stdout, out[-4000:]
