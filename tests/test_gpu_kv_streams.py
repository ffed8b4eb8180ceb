"""Memory of the layer over the 8-bit K/V tile cache when steps run on streams
other than the one that it was allocated on."""
import pytest
import torch

from block_sparse_attention_24_b200.stream import VedaStream
from tests.test_gpu_kv_cache import DEV, bf16

pytestmark = pytest.mark.gpu


def spans(tensors):
    return [(t.untyped_storage().data_ptr(), t.untyped_storage().data_ptr() + t.untyped_storage().nbytes()) for t in tensors]


@pytest.mark.parametrize("keep", [None, 2])
@pytest.mark.parametrize("explicit", [True, False])
def test_a_dropped_layers_memory_waits_for_its_steps(keep, explicit):
    """The cache is the default stream's, one workspace too; the last step runs
    on another stream, behind some work, when the layer goes."""
    n = 70
    q, k = bf16(1, 1, n, 4, 64), bf16(2, 1, n, 2, 64)
    want = None
    for drop in (False, True):
        layer = VedaStream(1, 4, 2, 64, 64, 4000, DEV, keep=keep)
        layer.step(q, k, k)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
            if not explicit:
                got = layer.step(q, k, k)
        if explicit:
            got = layer.step(q, k, k, stream=side)
        if not drop:
            side.synchronize()
            want = got
            continue
        held = [*layer.cache.tensors(), *layer._ws.values()]
        taken, sizes = spans(held), [t.untyped_storage().nbytes() for t in held]
        assert len(layer._ws) >= 1
        del layer, held
        new = [torch.full((x,), 0xff, dtype=torch.uint8, device=DEV) for x in sizes for _ in range(2)]
        for a0, a1 in spans(new):
            assert all(a1 <= b0 or b1 <= a0 for b0, b1 in taken)
        side.synchronize()
        assert torch.equal(got, want)


def test_a_reset_on_another_stream_holds_the_counts():
    layer = VedaStream(1, 4, 2, 64, 64, 4000, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    layer.reset(stream=side)
    held = [layer.cache.len, layer.cache.next_pos]
    taken, sizes = spans(held), [t.untyped_storage().nbytes() for t in held]
    del layer, held
    new = [torch.empty((x,), dtype=torch.uint8, device=DEV) for x in sizes for _ in range(2)]
    for a0, a1 in spans(new):
        assert all(a1 <= b0 or b1 <= a0 for b0, b1 in taken)
    side.synchronize()


@pytest.mark.parametrize("n", [1, 40])
def test_captured_steps_of_the_layer(n):
    """A workspace that is allocated while a step is captured serves replays
    and eager steps, in turn, and the layer can go when they are through."""
    q, k = [bf16(10 + i, 1, n, 4, 64) for i in range(6)], [bf16(20 + i, 1, n, 2, 64) for i in range(6)]
    make = lambda: VedaStream(1, 4, 2, 64, 64, 640, DEV, keep=4)
    e, a = make(), make()
    want = [e.step(x, y, y).clone() for x, y in zip(q, k)]      # loads every kernel before the capture
    qs, ks, o = q[0].clone(), k[0].clone(), torch.zeros_like(q[0])
    gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(gr, stream=side):
        a.step(qs, ks, ks, out=o)
    for i, (x, y) in enumerate(zip(q, k)):
        if i % 3 == 2:
            got = a.step(x, y, y)
        else:
            qs.copy_(x), ks.copy_(y)
            gr.replay()
            got = o
        assert torch.equal(got, want[i])
    a.check_status()
    torch.cuda.synchronize()
    del gr, a
    torch.cuda.synchronize()
    assert torch.zeros(1 << 20, device=DEV).sum().item() == 0
