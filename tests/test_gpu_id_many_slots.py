"""Experts' products of almost 2^31 slots on a GB300: places, tiles and rows past 31 bits."""
import pytest

from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOKEN, SLOT = 1, 0


@pytest.fixture(scope="module")
def rg():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_weight_out_gb300 import binding
    binding.load()
    return binding


def test_almost_2_31_slots(rg):
    """8 slots a token, half of them each of two experts, 8 x 8 weights; the last tiles end within a step of 2^31."""
    per, tokens = 8, (1 << 28) - 1
    slots = per * tokens
    need = slots * (4 + 16 + 16) + tokens * 16  # order, the result and the input's copy, the input
    if torch.cuda.mem_get_info()[0] < need + (40 << 30):
        pytest.skip("needs 120 GB of free device memory")
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(tokens, 8, generator=g, device=dev, dtype=torch.bfloat16)
    W = torch.randn(2, 8, 8, generator=g, device=dev).bfloat16()
    # slots by expert: the even ones, then the odd ones
    order = torch.empty(slots, dtype=torch.int32, device=dev)
    half = slots // 2
    torch.arange(0, slots, 2, dtype=torch.int32, device=dev, out=order[:half])
    torch.arange(1, slots, 2, dtype=torch.int32, device=dev, out=order[half:])
    start = torch.tensor([0, half, slots], dtype=torch.int32, device=dev)
    batch = rg.id_batch(2, per, start, order)
    y = torch.full((slots, 8), float("nan"), dtype=torch.bfloat16, device=dev)
    size = rg.rg_mul_mat_id_workspace_bytes(inputs.BF16, 8, 8, batch, SLOT)
    work = torch.empty(size, dtype=torch.uint8, device=dev)
    s = torch.cuda.current_stream()
    rg.check(rg.rg_mul_mat_id_ws(inputs.BF16, W, 8, 8, batch, inputs.BF16, x, 8, TOKEN, y, 8, SLOT, None, 0.0, work, size,
                                 s))
    assert rg.rg_check(s) == rg.RG_OK
    del work, order
    # eight exact products in F32 (at most 8 half steps of the sum of magnitudes), rounded once to bf16
    both = W.float().reshape(16, 8).T.contiguous()
    step = 1 << 23
    for t in range(0, tokens, step):
        a = x[t:t + step].float()
        ref, mag = (a[:, :, None] * both).sum(1), (a.abs()[:, :, None] * both.abs()).sum(1)
        ref, mag = ref.view(-1, 2, 8)[:, None], mag.view(-1, 2, 8)[:, None]
        got = y[t * per:(t + step) * per].view(-1, per // 2, 2, 8).float()
        assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + 2.0 ** -20 * mag).all())
    del x, y
    torch.cuda.empty_cache()
