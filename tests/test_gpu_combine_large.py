"""The combination of rows with an output of more 16-byte units than one launch
has threads (2^32): every token of it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("residual", [False, True])
def test_more_units_than_threads_in_a_launch(residual):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4a4_rank_corrected_amd as S
    t, n, k = 4100, 1 << 22, 2  # 4100 * 2^20 units of four fp32 columns
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < t * n * 4 + (8 << 30):
        pytest.skip("needs 77 GB of free device memory")
    print(f"combine t={t} n={n} residual={residual}", flush=True)
    rng = np.random.default_rng(5)
    rows = torch.randint(-64, 65, (3, n), device="cuda").float()
    index = torch.from_numpy(rng.integers(-1, 4, (t, k)).astype(np.int32)).cuda()
    weight = torch.from_numpy((rng.integers(-8, 9, (t, k)) / 4).astype(np.float32)).cuda()
    y = torch.full((t, n), 0.5 if residual else float("nan"), device="cuda")
    S.svdq_combine_rows(rows, index, weight, residual=y if residual else None, y=y)
    torch.cuda.synchronize()
    # multiples of 1/4 below 2^24 / 4: exact in any order
    live = ((index >= 0) & (index < 3)).float() * weight
    pick = index.clamp(0, 2).long()
    add = 0.5 if residual else 0.0
    cols = torch.tensor([0, 1, 4097, n // 2, n - 1], device="cuda")
    want = (rows[:, cols][pick] * live.unsqueeze(-1)).sum(1) + add
    assert torch.equal(y[:, cols], want)
    for i in (0, 1, 4094, 4095, 4096, t - 1):
        assert torch.equal(y[i], (rows[pick[i]] * live[i].unsqueeze(1)).sum(0) + add), i
    del y
    torch.cuda.empty_cache()
