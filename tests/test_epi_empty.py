"""Products with an epilogue of an empty batch: the binding takes the arguments
that it documents for any batch (CPU), and the calls return empty (GPU)."""
import pytest

from tests.test_epi_cpu import _Fake, _lib

torch = pytest.importorskip("torch")
S = pytest.importorskip("w4a4_rank_corrected_amd")
from w4a4_rank_corrected_amd import _binding as B  # noqa: E402

bf = torch.bfloat16


def _call(b=0, **kw):
    d = dict(y=_Fake((b, 64), bf), out_dtype=None, act="none", act_begin=0)
    d.update(kw)
    return B._epilogue(b, 64, torch.device("cuda:0"), **d)


def test_gates_of_an_empty_batch():
    _lib()
    for rows, gate_rows in ((1, None), (1, 0), (0, None), (0, 0), (0, 5)):  # one shared row, or no rows at all
        _, _, e = _call(gate=_Fake((rows, 64), bf), gate_rows=gate_rows, residual=_Fake((0, 64), bf))
        assert e.gate_rows == 0
    for shape, gate_rows in (((2, 64), None), ((1, 63), None), ((1, 64), 5)):
        with pytest.raises(ValueError, match="gate has shape"):
            _call(gate=_Fake(shape, bf), gate_rows=gate_rows)
    with pytest.raises(ValueError, match="gate has dtype"):
        _call(gate=_Fake((1, 64), torch.float32))
    _, _, e = _call(b=4, gate=_Fake((1, 64), bf))
    assert e.gate_rows == 4
    for rows in (0, 4):
        with pytest.raises(ValueError, match="gate has shape"):
            _call(b=4, gate=_Fake((rows, 64), bf))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int4", "w8a8", "fp4"])
def test_empty_batch_with_a_gate(fmt):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"empty {fmt}", flush=True)
    n, m, rank = 20, 64, 4
    e = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")
    f16, l1, l2 = torch.float16, e(rank, m, dt=bf), e(n, rank, dt=bf)
    x, gate, res, z = e(0, m, dt=bf), e(1, n, dt=bf), e(0, n, dt=bf), e(0, rank, dt=torch.float32)
    if fmt == "int4":
        layer = S.DeviceLayer.from_tensors(m, n, rank, e(1, n, 32), e(1, n, dt=f16), l1, l2)
        ops = e(1, 0, 32), e(1, 0, dt=f16), z
        gemm, linear = S.svdq_gemm_w4a4_lowrank_up_epi, S.svdq_linear_epi
    elif fmt == "w8a8":
        layer = S.DeviceLayer8.from_tensors(m, n, rank, e(1, n, 64, dt=torch.int8), e(n, dt=f16), l1, l2)
        ops = e(1, 0, 64, dt=torch.int8), e(0, dt=f16), z
        gemm, linear = S.svdq_w8a8_gemm_lowrank_up_epi, S.svdq_w8a8_linear_epi
    else:
        layer = S.DeviceLayerFp4.from_tensors(m, n, rank, 1.0, 1.0, e(1, n, 32), e(1, n, 4), l1, l2)
        ops = e(1, 0, 32), e(1, 0, 4), z
        gemm, linear = S.svdq_fp4_gemm_lowrank_up_epi, S.svdq_fp4_linear_epi
    for y in (gemm(*ops, layer, act="silu", gate=gate, residual=res), linear(x, layer, gate=gate, residual=res),
              linear(x, layer, gate=gate[:0], gate_rows=7, residual=res)):
        assert y.shape == (0, n) and y.dtype == bf
