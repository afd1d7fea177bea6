"""Two handles at once: what one needs must not be taken from the other.  The
limit of a kernel's dynamic shared memory is the device's, so a later handle
that needs less than an earlier one must not lower it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hiddens", [(3696, 7168), (7168, 3696), (7168, 64)])
def test_dispatch_of_the_first_after_the_second_is_made(hiddens):
    import combine_ep_layout_04_gb300 as ep
    layers = [ep.EpLayer(4, 256, h, 32, 8) for h in hiddens]
    idx = torch.rand(1024, 32, device="cuda").topk(8, -1).indices.int()
    for layer, h in zip(layers, hiddens):
        x = torch.randn(1024, h, device="cuda").to(torch.bfloat16)
        lay = layer.layout(idx)
        recv = layer.dispatch(x, lay)
        xl = layer.expert_layout(idx, torch.ones(1024, 8, device="cuda"), lay)
        assert torch.equal(recv, x[xl.recv_src_token.long()])
        assert layer.device_status() == 0
    for layer in layers:
        layer.close()


@pytest.mark.parametrize("experts", [(2048, 1536), (4096, 2560)])
def test_expert_layout_of_the_first_after_the_second_is_made(experts):
    import combine_ep_layout_04_gb300 as ep
    layers = [ep.EpLayer(2, 64, 64, e, 4) for e in experts]
    for layer, e in zip(layers, experts):
        idx = torch.rand(128, e, device="cuda").topk(4, -1).indices.int()
        lay = layer.layout(idx)
        xl = layer.expert_layout(idx, torch.ones(128, 4, device="cuda"), lay)
        assert torch.equal(xl.expert_count.long(), torch.bincount(idx.flatten().long(), minlength=e))
        assert layer.device_status() == 0
    for layer in layers:
        layer.close()
