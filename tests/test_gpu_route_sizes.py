"""Router: sizes beyond the limits are refused before anything of them is allocated."""
import pytest

from test_gpu_route import env  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_refused_before_anything_is_allocated(env):  # noqa: F811
    torch, pmx = env
    z = torch.randn(1 << 20, 8, device="cuda")
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for top in (9, 17, 1 << 20, (1 << 31) - 1):
        with pytest.raises(pmx.PmxError):
            pmx.route(z, top)
    assert torch.cuda.max_memory_allocated() == before
