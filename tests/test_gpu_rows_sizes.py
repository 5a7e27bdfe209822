"""As many tokens as the header allows, on the GPU."""
import pytest

pytestmark = pytest.mark.gpu


def test_two_thousand_million_rows_of_a_byte():
    """2^31 - 1 tokens in reverse and back: warps by the 2^28, offsets past 2^31."""
    import torch
    import counted_notify_sync_gb300 as cns
    cns.build()
    torch.cuda.set_device(0)
    n = 2 ** 31 - 1
    route = cns.new_route(8, 4, 1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randint(0, 256, (n, 1), generator=gen, device="cuda", dtype=torch.uint8)
    places = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32).view(n, 1)
    rows = torch.empty_like(x)
    assert cns.run_dispatch(route, x, places=places, rows=rows) is rows
    assert torch.equal(rows.flip(0), x)
    back = cns.run_dispatch(route, rows, places=places, rows=torch.empty_like(x))
    assert torch.equal(back, x)
