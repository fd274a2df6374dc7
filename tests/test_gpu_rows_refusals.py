"""Numbers that size the outputs of the row calls, refused before anything is
allocated or enqueued."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [0, -1, -10 ** 12, 33, 1025, 10 ** 13])
def test_counts_out_of_range(count):
    import fine_grained_block_token_b200 as fp8
    z = torch.randn(8, 64, device="cuda")
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(fp8.Fp8blError) as e:
        fp8.route(z, count)
    assert e.value.status == 2
    if not 1 <= count <= 1024:
        with pytest.raises(fp8.Fp8blError) as e:
            fp8.group_rows(ids, count)
        assert e.value.status == 2
    with pytest.raises(TypeError):
        fp8.route(z, "2")
    with pytest.raises(TypeError):
        fp8.route(z, 2.0)
    with pytest.raises(TypeError):
        fp8.group_rows(ids, None)
    assert fp8.route(z, 32)[0].shape == (8, 32) and fp8.group_rows(ids, 1024)[0].shape == (1025,)
    fp8.check()
