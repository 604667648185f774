"""What gqa_shard_combine takes as outputs, lses and streams, and what it refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu
N, B, Q, H, D = 2, 3, 4, 8, 128


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


@pytest.fixture(scope="module")
def parts():
    g = torch.Generator().manual_seed(170)
    return (torch.randn(N, B, Q, H, D, generator=g).cuda(), torch.randn(N, B, Q, H, generator=g).cuda())


def new(*shape, dtype=torch.bfloat16):
    return torch.full(shape, 7.0, dtype=dtype, device="cuda")


def test_outputs_and_lses_of_other_types_shapes_and_strides_are_refused(mla, parts):
    part, lse = parts
    for out in (new(B, Q, H, D, dtype=torch.float32), new(B, Q, H, D, dtype=torch.float16),
                new(B, Q, H, D).view(torch.int16)):
        with pytest.raises(TypeError):
            mla.gqa_shard_combine(part, lse, out=out)
        assert bool((out == out.flatten()[0]).all())          # nothing was written
    for out in (new(B, H, Q, D), new(B, H, Q, D).transpose(1, 2), new(B, Q, H, 2 * D)[..., :D],
                new(B - 1, Q, H, D), new(B * Q * H * D - 1)):
        with pytest.raises(ValueError):
            mla.gqa_shard_combine(part, lse, out=out)
    with pytest.raises(TypeError):
        mla.gqa_shard_combine(part, lse, lse_out=new(B, Q, H))
    for l in (new(B, H, Q, dtype=torch.float32), new(B, Q, 2 * H, dtype=torch.float32)[..., ::2],
              new(B * Q * H - 1, dtype=torch.float32)):
        with pytest.raises(ValueError):
            mla.gqa_shard_combine(part, lse, lse_out=l)
    for l in (lse.transpose(2, 3).contiguous(), lse[:1], lse.transpose(2, 3)):
        with pytest.raises(ValueError):
            mla.gqa_shard_combine(part, l)


def test_outputs_with_room(mla, parts):
    part, lse = parts
    want, want_lse = mla.gqa_shard_combine(part, lse)
    for out, l in ((new(B, Q, H, D), new(B, Q, H, dtype=torch.float32)),
                   (new(B + 2, Q, H, D), new(B + 1, Q, H, dtype=torch.float32)),
                   (new(B * Q, H * D), new(B * Q * H + 5, dtype=torch.float32))):
        got, got_lse = mla.gqa_shard_combine(part, lse, out=out, lse_out=l)
        assert got is out and got_lse is l
        assert torch.equal(out.flatten()[:want.numel()], want.flatten())
        assert torch.equal(l.flatten()[:want_lse.numel()], want_lse.flatten())
        assert bool((out.flatten()[want.numel():] == 7).all())
        assert bool((l.flatten()[want_lse.numel():] == 7).all())


class Handle:
    """A stream of another library: all it has is the CUDA handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


def test_streams_known_by_their_handle(mla, parts):
    part, lse = parts
    want = mla.gqa_shard_combine(part, lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, Handle(side.cuda_stream), torch.cuda.ExternalStream(side.cuda_stream),
              Handle(torch.cuda.default_stream().cuda_stream), torch.cuda.default_stream()):
        got = mla.gqa_shard_combine(part, lse, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    for s in (3, "stream", object()):
        with pytest.raises(AttributeError):
            mla.gqa_shard_combine(part, lse, stream=s)


def test_work_is_on_the_stream_of_the_handle(mla, parts):
    """The call is captured into a graph of the handle's stream."""
    part, lse = parts
    want = mla.gqa_shard_combine(part, lse)
    out, l = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        mla.gqa_shard_combine(part, lse, out=out, lse_out=l, stream=Handle(side.cuda_stream))
    assert bool((out == 0).all())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(l, want[1])
